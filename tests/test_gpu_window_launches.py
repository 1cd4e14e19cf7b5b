"""Launch forms of the windowed calls: calls one behind the other, captured
ones, and ones beside each other on two streams, for both of the decode
step's forms and for chunks."""
import numpy as np
import pytest
import torch

import decode_attention_dq_b200 as dq
from tests.test_gpu_window import BF16, F32, _decode, _ints, _np, _prefill, _rounded, _setup, _workspace

pytestmark = pytest.mark.gpu


def test_calls_with_different_tables_one_behind_the_other():
    # Clusters of one call take the place of those of the call before it, whose tables are others.
    B, Hkv, G, T = 40, 2, 4, 300
    sets = []
    for bits, v_levels in ((1.96, 6), (2.26, 8), (3.0, 4)):
        w, lib, _, kc, vc, _, _ = _setup(B, Hkv, G, T, bits, v_levels)
        q = torch.from_numpy(dq.synth.q_block(w)).cuda()
        lens, ws, stats = _ints([300 - 7 * b for b in range(B)]), _workspace(lib, B, Hkv * G, Hkv, T), dq.new_stats()
        outs = [torch.empty_like(q) for _ in range(12)]
        sets.append((lib, q, kc, vc, lens, ws, stats, outs))
    want = []
    for lib, q, kc, vc, lens, ws, stats, outs in sets:
        out = torch.empty_like(q)
        dq.dq_decode_attention_window(lib, q, kc, vc, lens, T, 100, 4, out, ws)
        torch.cuda.synchronize()
        want.append(out)
    for i in range(12):
        for lib, q, kc, vc, lens, ws, stats, outs in sets:
            dq.dq_decode_attention_window(lib, q, kc, vc, lens, T, 100, 4, outs[i], ws, stats=stats)
    for (_, _, _, _, _, _, stats, outs), out in zip(sets, want):
        assert all(torch.equal(x, out) for x in outs)
        s = dq.stats_dict(stats)
        assert s["integrity_errors"] == 0 and s["wait_timeouts"] == 0
