"""Launch forms of the windowed calls: calls one behind the other, captured
ones, and ones beside each other on two streams, for both of the decode
step's forms and for chunks."""
import ctypes

import numpy as np
import pytest
import torch

import decode_attention_dq_b200 as dq
from decode_attention_dq_b200 import synth
from tests import _common as cm
from tests import _pages as R
from tests import _window as W
from tests.test_gpu_window import BF16, F32, _decode, _ints, _np, _prefill, _rounded, _setup, _workspace

pytestmark = pytest.mark.gpu


def test_calls_with_different_tables_one_behind_the_other():
    # Clusters of one call take the place of those of the call before it, whose tables are others.
    B, Hkv, G, T = 40, 2, 4, 300
    sets = []
    for bits, v_levels in ((1.96, 6), (2.26, 8), (3.0, 4)):
        w, lib, _, kc, vc, _, _ = _setup(B, Hkv, G, T, bits, v_levels)
        q = torch.from_numpy(synth.q_block(w)).cuda()
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
    q = _rounded(synth.q_block(w), BF16)
    got = _np(_decode(lib, q, kc, vc, lens, 2 ** 40, 0, dtype=BF16))
    full = cm.gpu_attention(lib, q, kc, vc, lens, T_max=kc.shape[2], q_dtype=BF16, out_dtype=BF16)
    want, bound = (x[:, 0] for x in W.attention(ref, q[:, None], rk, rv, np.array(lens) - 1, T, 0, chunk=False))
    W.assert_within(got, want, bound, True, "windowed")
    W.assert_within(full, want, bound, True, "without a window")
    assert np.all(np.abs(got - full) <= 2 * bound + 2.0 ** -7 * (np.abs(want) + bound))


def _captured(call):
    """A graph of one call, after one that is not captured."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    return graph


@pytest.mark.parametrize("B", [3, 60])  # clusters; prefix, split and combine kernels launched ahead
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_captured_decode_steps_follow_lengths_and_queries(B, dtype):
    Hkv, G, T = 4, 2, 500
    w, lib, _, kc, vc, _, _ = _setup(B, Hkv, G, T)
    q = synth.q_block(w)
    qt, seq = torch.from_numpy(q).cuda().to(dtype), _ints([1] * B)
    out, ws = torch.empty_like(qt), _workspace(lib, B, Hkv * G, Hkv, T)
    after = torch.empty_like(out)

    def call():  # two steps that share the workspace, and a kernel that reads what they wrote
        dq.dq_decode_attention_window(lib, qt, kc, vc, seq, T, 60, 3, out, ws)
        dq.dq_decode_attention_window(lib, qt, kc, vc, seq, T, 130, 40, after, ws)
        after.add_(out)

    graph = _captured(call)
    for step in range(4):
        lens = [(b * 37 + 113 * step) % (T + 1) for b in range(B)]
        seq.copy_(_ints(lens))
        qt.copy_(torch.from_numpy(q * (1 + step)))
        graph.replay()
        torch.cuda.synchronize()
        first = _decode(lib, _np(qt).astype(np.float32), kc, vc, lens, 60, 3, dtype=dtype)
        second = _decode(lib, _np(qt).astype(np.float32), kc, vc, lens, 130, 40, dtype=dtype)
        assert torch.equal(out, first) and torch.equal(after, second + first)


@pytest.mark.parametrize("own_workspace", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_captured_chunks_follow_their_positions(own_workspace, dtype):
    B, Hkv, G, T, n_q = 3, 2, 4, 700, 90
    w, lib, _, kc, vc, _, _ = _setup(B, Hkv, G, T)
    q, start = synth.q_chunk(w, n_q), _ints([0] * B)
    qt = torch.from_numpy(q).cuda()
    out = torch.empty(q.shape, dtype=dtype, device="cuda")
    need = dq.dq_prefill_window_workspace_bytes(lib, B, Hkv, kc.shape[2], n_q, 100, 5)
    ws = None if own_workspace else torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    graph = _captured(lambda: dq.dq_prefill_attention_window(lib, qt, kc, vc, start, 100, 5, out, workspace=ws))
    for at in ([600, 0, 77], [-3, 650, 610], [128, 900, 300]):
        start.copy_(_ints(at))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, _prefill(lib, q, kc, vc, at, 100, 5, out_dtype=dtype))


def test_chunks_and_balanced_decode_steps_on_two_streams():
    B, Hkv, G, T = 60, 4, 2, 400
    w, lib, _, kc, vc, _, _ = _setup(B, Hkv, G, T)
    n_q, q1, qc = 33, synth.q_block(w), synth.q_chunk(w, 33)
    lens, start = [400 - 5 * b for b in range(B)], [300 - 5 * b for b in range(B)]
    a, b = _decode(lib, q1, kc, vc, lens, 100, 4), _prefill(lib, qc, kc, vc, start, 100, 4)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(10):
        with torch.cuda.stream(s1):
            x = [_decode(lib, q1, kc, vc, lens, 100, 4) for _ in range(2)]
        with torch.cuda.stream(s2):
            y = [_prefill(lib, qc, kc, vc, start, 100, 4) for _ in range(2)]
        torch.cuda.synchronize()
        assert all(torch.equal(v, a) for v in x) and all(torch.equal(v, b) for v in y)


def test_captured_fork_compact_and_copies_follow_the_state():
    # Twelve rounds of one graph that forks, copies, compacts and copies, from state to state.
    Hkv, P, B, mp = 2, 150, 6, 12
    lib = cm.lib_tables(Hkv)
    rng = np.random.default_rng(4)
    refs, table, lens = R.random_state(rng, P, B, mp)
    kp, vp = (torch.randint(0, 256, (3, P, Hkv, 36, 32), dtype=torch.uint8, device="cuda") for _ in range(2))
    r, t, L = (torch.as_tensor(x, dtype=torch.int32).cuda() for x in (refs, table, lens))
    mid, parent = [torch.empty_like(x) for x in (r, t, L)], _ints(list(range(B)))
    pairs, moves = _ints([[0, 0]] * B), _ints([[0, 0]] * (P // 2))
    c1, c2 = dq.new_page_counts(), dq.new_page_counts()
    ws = torch.full((dq.dq_pages_workspace_bytes(lib, P, B, mp),), 0xA5, dtype=torch.uint8, device="cuda")

    def call():
        dq.dq_pages_fork(lib, r, t, L, parent, *mid, pairs, c1, ws)
        dq.dq_pages_copy(lib, kp, vp, pairs, c1)
        dq.dq_pages_compact(lib, mid[0], mid[1], r, t, moves, c2, ws)
        dq.dq_pages_copy(lib, kp, vp, moves, c2)
        L.copy_(mid[2])

    keep = [x.clone() for x in (r, t, L, kp, vp)]
    graph = _captured(call)
    for x, y in zip((r, t, L, kp, vp), keep):
        x.copy_(y)
    kw, vw = (x.cpu().numpy().copy() for x in (kp, vp))
    for step in range(12):
        more = rng.integers(-1, B, B) if step % 3 else np.arange(B)
        parent.copy_(_ints(more.tolist()))
        graph.replay()
        refs, table, lens, p1, w1 = R.fork(refs, table, lens, more)
        refs, table, p2, w2 = R.compact(refs, table)
        for todo, n in ((p1, w1["pairs"]), (p2, w2["pairs"])):
            for s, d in todo[:n]:
                kw[:, d], vw[:, d] = kw[:, s], vw[:, s]
        assert dq.page_counts_dict(c1) == w1 and dq.page_counts_dict(c2) == w2
        for got, want in ((r, refs), (t, table), (L, lens), (pairs, p1), (moves, p2), (kp, kw), (vp, vw)):
            np.testing.assert_array_equal(got.cpu().numpy(), np.asarray(want))


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_a_query_that_is_not_finite_gives_zero_and_stays_with_its_row(value):
    Hkv, G, T = 2, 4, 300
    for B in (4, 80):
        w, lib, ref, kc, vc, rk, rv = _setup(B, Hkv, G, T)
        lens, q = [300, 33, 1, 64] * (B // 4), synth.q_block(w)
        bad = q.copy()
        bad[[0, 1, 2], [1, 7, 0], 5] = value
        want = _decode(lib, q, kc, vc, lens, 100, 4).clone()
        want[[0, 1, 2], [1, 7, 0]] = 0.0
        assert torch.equal(_decode(lib, bad, kc, vc, lens, 100, 4), want)
    q = synth.q_chunk(w, 70)[:2]
    bad = q.copy()
    rows = ([0, 0, 1], [0, 33, 69], [0, 5, 7])
    bad[(*rows, 9)] = value
    want, bound = W.attention(ref, q, rk[:2], rv[:2], [230, 0], 100, 4, chunk=True)
    want[rows], bound[rows] = 0.0, 0.0
    W.assert_within(_np(_prefill(lib, bad, kc[:2].contiguous(), vc[:2].contiguous(), [230, 0], 100, 4)), want, bound, False,
                    "chunk")


def test_a_call_that_failed_does_not_fail_the_next_one():
    # A call into a stream whose capture has been broken is refused by the runtime; the next call on another stream,
    # whose launches ask for the last error, succeeds.
    rt = ctypes.CDLL("libcudart.so.12")
    lib = cm.lib_tables(2)
    r, t, L = dq.new_page_state(8, 2, 4)
    counts, ws = dq.new_page_counts(), torch.empty(dq.dq_pages_workspace_bytes(lib, 8, 2, 4), dtype=torch.uint8, device="cuda")
    cache = dq.new_cache(1, 2, 32, 36)
    k, zero = torch.randn(1, 2, 4, 128, device="cuda"), _ints([0])
    seq, q = _ints([4]), torch.randn(1, 2, 128, device="cuda")
    out, dws = torch.empty_like(q), _workspace(lib, 1, 2, 2, 32)
    side, graph = torch.cuda.Stream(), ctypes.c_void_p()
    torch.cuda.synchronize()
    assert rt.cudaStreamBeginCapture(ctypes.c_void_p(side.cuda_stream), 0) == 0
    try:
        assert rt.cudaDeviceSynchronize() != 0  # (not allowed while a stream is captured: the capture is broken)
        with pytest.raises(dq.DqError):
            dq.dq_pages_advance(lib, r, t, L, L, r, t, L, counts, ws, stream=side)
        with pytest.raises(dq.DqError):
            dq.dq_decode_attention_window(lib, q, cache, cache, seq, 32, 8, 0, out, dws, stream=side)
    finally:
        rt.cudaStreamEndCapture(ctypes.c_void_p(side.cuda_stream), ctypes.byref(graph))
        rt.cudaGetLastError()
    dq.dq_append_kv(lib, k, k, zero, cache, cache.clone(), workspace=False)
    dq.dq_pages_advance(lib, r, t, L, _ints([1, 1]), r, t, L, counts, ws)
    assert L.tolist() == [1, 1]
