"""Launch forms of the windowed calls: calls one behind the other, captured
ones, and ones beside each other on two streams, for both of the decode
step's forms and for chunks."""
import numpy as np
import pytest
import torch

import decode_attention_dq_b200 as dq
from tests import _common as cm
from tests import _window as W
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


@pytest.mark.parametrize("B,Hkv,T", [(1, 8, 1100), (40, 8, 170)])  # a cluster per (b, h); the balanced split
def test_a_window_of_everything_agrees_but_for_the_order_of_sums(B, Hkv, T):
    # Both calls are within the bound of the definition; so they differ by two bounds and a bf16 step at most.
    G = 4
    w, lib, ref, kc, vc, rk, rv = _setup(B, Hkv, G, T)
    lens = [max(1, T - 9 * b) for b in range(B)]
    q = _rounded(dq.synth.q_block(w), BF16)
    got = _np(_decode(lib, q, kc, vc, lens, 2 ** 40, 0, dtype=BF16))
    full = cm.gpu_attention(lib, q, kc, vc, lens, T_max=kc.shape[2], q_dtype=BF16, out_dtype=BF16)
    want, bound = (x[:, 0] for x in W.attention(ref, q[:, None], rk, rv, np.array(lens) - 1, T, 0, chunk=False))
    W.assert_within(got, want, bound, True, "windowed")
    W.assert_within(full, want, bound, True, "without a window")
    assert np.all(np.abs(got - full) <= 2 * bound + 2.0 ** -7 * (np.abs(want) + bound))
