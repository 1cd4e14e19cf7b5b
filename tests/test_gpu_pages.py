"""dq_pages_advance, _fork, _compact and _copy against their definitions
(tests/_pages.py): every output a whole number and equal. Pools from one page
to several hundred thousand, tables of one entry and of more than a segment,
shared and foreign references, pools that run short, entries, parents and
lengths out of range, outputs that are the inputs, captured and repeated
calls; then the calls together with the append and the windowed attention."""
import numpy as np
import pytest
import torch

import decode_attention_dq_b200 as dq
from decode_attention_dq_b200 import synth
from tests import _common as cm
from tests import _pages as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tab():
    return cm.lib_tables(2)


def _ints(v):
    return torch.as_tensor(np.ascontiguousarray(v), dtype=torch.int32).cuda()


def _workspace(tab, P, B, mp):
    ws = torch.empty(dq.dq_pages_workspace_bytes(tab, P, B, mp), dtype=torch.uint8, device="cuda")
    return ws.fill_(0xA5)


def _same(got, want, what):
    for k, (g, w) in enumerate(zip(got, want)):
        if isinstance(w, dict):
            assert dq.page_counts_dict(g) == w, what
        else:
            np.testing.assert_array_equal(g.cpu().numpy(), np.asarray(w).reshape(g.shape), err_msg="%s, output %d" % (what, k))


def _advance(tab, refs, table, lens, n_new, window=0, sinks=0, in_place=False):
    B, mp = table.shape
    r, t, L = _ints(refs), _ints(table), _ints(lens)
    outs = (r, t, L) if in_place else tuple(torch.full_like(x, -77) for x in (r, t, L))
    counts = dq.new_page_counts().fill_(-5)
    dq.dq_pages_advance(tab, r, t, L, _ints(n_new), *outs, counts, _workspace(tab, len(refs), B, mp), window=window, sinks=sinks)
    return (*outs, counts)


SIZES = [(1, 1, 1), (3, 5, 1), (40, 6, 9), (700, 33, 40), (129, 1, 600), (6000, 7, 1100), (70001, 70, 513), (300000, 9, 33)]


@pytest.mark.parametrize("P,B,mp", SIZES)
@pytest.mark.parametrize("in_place", [False, True])
def test_advance(tab, P, B, mp, in_place):
    rng = np.random.default_rng(P + B + mp)
    for window, sinks in ((0, 0), (1, 0), (40, 4), (33, 64), (32 * mp, 5)):
        refs, table, lens = R.random_state(rng, P, B, mp, window=window, sinks=sinks)
        n = rng.choice([-1, 0, 1, 1, 1, 31, 32, 33, 200, 32 * mp], B)
        _same(_advance(tab, refs, table, lens, n, window, sinks, in_place), R.advance(refs, table, lens, n, window, sinks),
              "window %d sinks %d" % (window, sinks))


@pytest.mark.parametrize("in_place", [False, True])
def test_advance_of_a_large_state(tab, in_place):
    # More counts and entries than one launch takes: the rows go on all SMs.
    rng = np.random.default_rng(5)
    P, B, mp = 660001, 30, 701
    for window, sinks in ((0, 0), (900, 40)):
        refs, table, lens = R.random_state(rng, P, B, mp, window=window, sinks=sinks)
        table[3, 5], table[4, 6], lens[7] = P, -9, -50
        refs[:200000] = 1
        n = rng.choice([-1, 0, 1, 33, 200, 9000], B)
        _same(_advance(tab, refs, table, lens, n, window, sinks, in_place), R.advance(refs, table, lens, n, window, sinks),
              "window %d sinks %d" % (window, sinks))


def test_advance_hands_out_what_it_takes_back(tab):
    # A full pool: rows 0 and 2 end, row 1 grows into their pages.
    table = np.array([[5, 4, -1, -1], [1, -1, -1, -1], [0, 2, 3, -1]])
    refs = np.ones(6)
    got = _advance(tab, refs, table, [64, 20, 70], [-1, 100, -1])
    _same(got, ([1, 1, 1, 1, 0, 0], [[-1] * 4, [1, 0, 2, 3], [-1] * 4], [0, 120, 0],
                dict(free_pages=2, taken=3, released=5, short_of=0, bad=0, clamped=0, pairs=0, reserved=0)), "full pool")


def test_many_short_rows(tab):
    # More rows than a CTA's part is wide.
    rng = np.random.default_rng(2)
    P, B, mp = 30000, 18000, 2
    refs, table, lens = R.random_state(rng, P, B, mp)
    n = rng.choice([-1, 0, 1, 1, 40], B)
    _same(_advance(tab, refs, table, lens, n), R.advance(refs, table, lens, n), "advance")
    parent = rng.integers(-1, B, 20000)
    _same(_fork(tab, refs, table, lens, parent), R.fork(refs, table, lens, parent), "fork")
    _same(_compact(tab, refs, table), R.compact(refs, table), "compact")


def test_arrays_that_start_anywhere(tab):
    # Four-byte aligned views: no 16-byte accesses.
    rng = np.random.default_rng(3)
    P, B, mp = 5000, 12, 64

    def off(x):
        x = _ints(x)
        buf = torch.full((x.numel() + 1,), -77, dtype=torch.int32, device="cuda")
        buf[1:] = x.reshape(-1)
        return buf[1:].view(x.shape)

    refs, table, lens = R.random_state(rng, P, B, mp)
    n, ws, c = rng.choice([-1, 1, 90], B), _workspace(tab, P, B, mp), dq.new_page_counts()
    o = [off(np.full_like(x, -77)) for x in (refs, table, lens)]
    dq.dq_pages_advance(tab, off(refs), off(table), off(lens), off(n), *o, c, ws)
    _same((*o, c), R.advance(refs, table, lens, n), "advance")
    pairs = off(np.zeros((B, 2)))
    parent = rng.integers(-1, B, B)
    o = [off(np.full_like(x, -77)) for x in (refs, table, lens)]
    dq.dq_pages_fork(tab, off(refs), off(table), off(lens), off(parent), *o, pairs, c, ws)
    _same((*o, pairs, c), R.fork(refs, table, lens, parent), "fork")
    o, pairs = [off(np.full_like(x, -77)) for x in (refs, table)], off(np.zeros((P // 2, 2)))
    dq.dq_pages_compact(tab, off(refs), off(table), *o, pairs, c, ws)
    _same((*o, pairs, c), R.compact(refs, table), "compact")


def test_advance_out_of_range(tab):
    # Lengths beyond the table and negative ones, entries that are no pages, a pool too small.
    table = np.array([[0, 99, -7], [1, 2, 3], [2 ** 31 - 1, -1, 4], [-2 ** 31, -1, -1]])
    refs = np.array([1, 1, 1, 1, 1, 0])
    lens, n = [2 ** 31 - 1, 90, -40, -1], [2 ** 31 - 1, 2 ** 31 - 1, 70, -2 ** 31]
    for window, sinks in ((0, 0), (20, 2 ** 50), (2 ** 60, 3)):
        _same(_advance(tab, refs, table, lens, n, window, sinks), R.advance(refs, table, lens, n, window, sinks), "out of range")


def test_a_row_without_new_tokens_keeps_what_its_last_one_sees(tab):
    # Length 65, window 33: the last token's query sees tokens 32 .. 64, the next one's 33 .. 65 and no longer page 0.
    table, refs = np.array([[4, 2, 0, -1]]), np.array([1, 0, 1, 0, 1])
    for n, left in ((0, [4, 2, 0, -1]), (1, [-1, 2, 0, -1]), (-1, [-1] * 4)):
        got = _advance(tab, refs, table, [65], [n], window=33)
        _same(got, R.advance(refs, table, [65], [n], 33), "n %d" % n)
        assert got[1].tolist() == [left]


def test_advance_of_no_rows_counts_the_pool(tab):
    got = _advance(tab, [0, 1, 0, 0], np.zeros((0, 3)), [], [])
    _same(got, ([0, 1, 0, 0], np.zeros((0, 3)), [], dict.fromkeys(dq._native.PAGE_COUNT_FIELDS, 0) | dict(free_pages=3)), "no rows")


def _fork(tab, refs, table, lens, parent):
    B, mp = table.shape
    n = len(parent)
    r, t, L = _ints(refs), _ints(table), _ints(lens)
    outs = (torch.full_like(r, -77), torch.full((n, mp), -77, dtype=torch.int32, device="cuda"),
            torch.full((n,), -77, dtype=torch.int32, device="cuda"), torch.full((n, 2), -77, dtype=torch.int32, device="cuda"))
    counts = dq.new_page_counts()
    dq.dq_pages_fork(tab, r, t, L, _ints(parent), *outs, counts, _workspace(tab, len(refs), max(B, n), mp))
    return (*outs, counts)


@pytest.mark.parametrize("P,B,mp", SIZES)
def test_fork(tab, P, B, mp):
    rng = np.random.default_rng(P + B + mp)
    refs, table, lens = R.random_state(rng, P, B, mp)
    for parent in (np.arange(B), rng.integers(-1, B, B), np.full(B + 3, B - 1), rng.integers(-2, B + 2, 4 * B), np.full(2, -1),
                   rng.integers(0, B, 2500)):
        _same(_fork(tab, refs, table, lens, parent), R.fork(refs, table, lens, parent), "parents %s" % parent[:8])


def test_fork_out_of_range_and_from_nothing(tab):
    table = np.array([[0, 99, -7], [1, 2, 3], [2 ** 31 - 1, -1, 4]])
    refs, lens = np.array([1, 1, 1, 2, 1, 0]), [40, 2 ** 31 - 1, -5]
    parent = [0, 1, 1, 2 ** 31 - 1, -2 ** 31, 2, 0]
    _same(_fork(tab, refs, table, lens, parent), R.fork(refs, table, lens, parent), "out of range")
    empty = np.zeros((0, 3), dtype=np.int64)
    _same(_fork(tab, refs, empty, [], [0, -1]), R.fork(refs, empty, [], [0, -1]), "no old rows")
    _same(_fork(tab, refs, table, lens, []), R.fork(refs, table, lens, []), "no new rows")


def _compact(tab, refs, table, in_place=False):
    B, mp = table.shape
    r, t = _ints(refs), _ints(table)
    outs = (r, t) if in_place else (torch.full_like(r, -77), torch.full_like(t, -77))
    pairs = torch.full((max(1, len(refs) // 2), 2), -77, dtype=torch.int32, device="cuda")
    counts = dq.new_page_counts()
    dq.dq_pages_compact(tab, r, t, *outs, pairs, counts, _workspace(tab, len(refs), B, mp))
    return (*outs, pairs, counts)


@pytest.mark.parametrize("P,B,mp", SIZES)
@pytest.mark.parametrize("in_place", [False, True])
def test_compact(tab, P, B, mp, in_place):
    rng = np.random.default_rng(P + B + mp)
    refs, table, _ = R.random_state(rng, P, B, mp)
    _same(_compact(tab, refs, table, in_place), R.compact(refs, table), "random")
    for refs in (np.zeros(P), np.ones(P), np.r_[np.zeros(P // 2), np.ones(P - P // 2)], np.r_[np.ones(P - P // 2), np.zeros(P // 2)]):
        _same(_compact(tab, refs, table, in_place), R.compact(refs, table), "in blocks")


def test_compact_out_of_range_and_of_no_rows(tab):
    table, refs = np.array([[0, 99, -7], [1, 2, 3], [2 ** 31 - 1, -1, 4]]), np.array([0, 3, 0, -2, 1, 7])
    _same(_compact(tab, refs, table), R.compact(refs, table), "out of range")
    empty = np.zeros((0, 3), dtype=np.int64)
    _same(_compact(tab, refs, empty), R.compact(refs, empty), "no rows")


@pytest.mark.parametrize("bits,Hkv,layers", [(1.96, 1, 1), (2.26, 3, 5), (3.0, 8, 2)])
def test_copy(bits, Hkv, layers):
    t = cm.lib_tables(Hkv, bits, 2.26)
    P = 50
    g = torch.Generator(device="cuda").manual_seed(1)
    k = torch.randint(0, 256, (layers, P, Hkv, t.k.container_bytes, 32), dtype=torch.uint8, device="cuda", generator=g)
    v = torch.randint(0, 256, (layers, P, Hkv, t.v.container_bytes, 32), dtype=torch.uint8, device="cuda", generator=g)
    pairs = [(7, 3), (49, 0), (-1, -1), (12, 49 - 1), (50, 1), (2, -3), (2 ** 31 - 1, 5), (30, 31)]
    for n in (None, 0, 2, 8, 100, -4):
        for one_layer in (False, True):
            kk, vv = k.clone(), v.clone()
            kw, vw = k.clone(), v.clone()
            counts, used = None, len(pairs)
            if n is not None:
                counts = dq.new_page_counts()
                counts[6] = n
                used = min(max(n, 0), len(pairs))
            done = [p for p in pairs[:used] if 0 <= p[0] < P and 0 <= p[1] < P]
            at = slice(layers - 1, layers) if one_layer else slice(None)
            for s, d in done:
                kw[at, d], vw[at, d] = k[at, s], v[at, s]
            stats = dq.new_stats()
            a, b = (kk[-1], vv[-1]) if one_layer else (kk, vv)
            dq.dq_pages_copy(t, a, b, _ints(pairs), counts, stats=stats)
            assert torch.equal(kk, kw) and torch.equal(vv, vw)
            assert dq.stats_dict(stats)["bad_pages"] == sum(p not in done and p != (-1, -1) for p in pairs[:used])


def test_copy_of_layers_that_are_apart(tab):
    P, layers = 20, 3
    k = torch.randint(0, 256, (2 * layers, P, 2, 36, 32), dtype=torch.uint8, device="cuda")
    v = torch.randint(0, 256, (layers, P, 2, 36, 32), dtype=torch.uint8, device="cuda")
    kw, vw = k.clone(), v.clone()
    kw[::2, 4], vw[:, 4] = k[::2, 19], v[:, 19]
    dq.dq_pages_copy(tab, k[::2], v, _ints([[19, 4]]))
    assert torch.equal(k, kw) and torch.equal(v, vw)


def test_copy_past_four_gigabytes():
    # A pool whose last page starts beyond 2^32 bytes.
    t = cm.lib_tables(8, 3.0, 3.0)
    page = 8 * 48 * 32
    P = 2 ** 32 // page + 10
    k = torch.empty((P, 8, 48, 32), dtype=torch.uint8, device="cuda")
    v = torch.empty_like(k)
    for p, x in ((P - 1, 11), (0, 22), (5, 33)):
        k[p], v[p] = x, x + 100
    dq.dq_pages_copy(t, k, v, _ints([[P - 1, 5], [0, P - 2]]))
    for pool, d in ((k, 0), (v, 100)):
        assert bool((pool[5] == 11 + d).all()) and bool((pool[P - 2] == 22 + d).all()) and bool((pool[P - 1] == 11 + d).all())


def test_argument_errors(tab):
    r, t, L = dq.new_page_state(8, 2, 4)
    c, ws, n = dq.new_page_counts(), _workspace(tab, 8, 2, 4), _ints([1, 1])
    pairs = torch.empty((2, 2), dtype=torch.int32, device="cuda")
    outs = [torch.empty_like(x) for x in (r, t, L)]
    with pytest.raises(dq.DqError, match="workspace"):
        dq.dq_pages_advance(tab, r, t, L, n, *outs, c, ws[:256])
    with pytest.raises(dq.DqError, match="shape"):
        dq.dq_pages_advance(tab, r, t, L, n, *outs, c, ws, window=-1)
    for bad in ((r, outs[1], outs[2]), (outs[0], t, outs[2]), (outs[0], outs[1], L)):
        with pytest.raises(dq.DqError, match="shape"):
            dq.dq_pages_fork(tab, r, t, L, n, *bad, pairs, c, ws)
    with pytest.raises(ValueError, match="pairs"):
        dq.dq_pages_compact(tab, r, t, r, t, pairs, c, ws)
    with pytest.raises(ValueError, match="lens"):
        dq.dq_pages_advance(tab, r, t, L.long(), n, *outs, c, ws)
    with pytest.raises(ValueError, match="pools"):
        dq.dq_pages_copy(tab, dq.new_pool(8, 3, 36), dq.new_pool(8, 2, 36), pairs)


def test_captured_steps_follow_the_state(tab):
    # Twenty decode steps of one graph, in place, against the definition.
    rng = np.random.default_rng(8)
    P, B, mp, window, sinks = 60, 6, 20, 50, 4
    refs, table, lens = R.random_state(rng, P, B, mp, window=window, sinks=sinks)
    r, t, L, n = _ints(refs), _ints(table), _ints(lens), _ints(np.zeros(B))
    counts, ws = dq.new_page_counts(), _workspace(tab, P, B, mp)
    call = lambda: dq.dq_pages_advance(tab, r, t, L, n, r, t, L, counts, ws, window=window, sinks=sinks)  # noqa: E731
    n.fill_(1)
    keep = [x.clone() for x in (r, t, L)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    for x, y in zip((r, t, L), keep):
        x.copy_(y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for step in range(20):
        more = rng.choice([-1, 0, 1, 1, 1, 40], B)
        n.copy_(_ints(more))
        graph.replay()
        want = R.advance(refs, table, lens, more, window, sinks)
        _same((r, t, L, counts), want, "step %d" % step)
        refs, table, lens = want[:3]


def test_serving_run():
    """Prompts in chunks, sampling by forks, decode steps, sequences that end and a compaction, behind page tables
    and a window; every attention output equals that of a contiguous cache holding the same tokens."""
    Hkv, G, window, sinks, mp, P = 2, 4, 70, 5, 16, 40
    tab = cm.lib_tables(Hkv)
    w = synth.scaled(synth.WORKLOADS["qwen3_8b_b16_t8k"], B=6, Hkv=Hkv, Hq=Hkv * G, T=32 * mp)
    K, V, _ = cm.inputs(w)
    K, V = (torch.from_numpy(x).cuda().bfloat16() for x in (K, V))
    kp, vp = dq.new_pool(P, Hkv, 36).fill_(0xFF), dq.new_pool(P, Hkv, 36).fill_(0xFF)
    refs, table, lens = dq.new_page_state(P, 6, mp)
    spare = dq.new_page_state(P, 6, mp)
    kc, vc = dq.new_cache(6, Hkv, 32 * mp, 36), dq.new_cache(6, Hkv, 32 * mp, 36)
    counts, ws = dq.new_page_counts(), _workspace(tab, P, 6, mp)
    stats = dq.new_stats()
    held = [0] * 6  # lengths on the host, for the test's own slicing

    def append(n):
        dq.dq_pages_advance(tab, refs, table, lens, _ints(n), refs, table, lens, counts, ws, window=window, sinks=sinks)
        got = dq.page_counts_dict(counts)
        assert got["short_of"] == 0 and got["bad"] == 0 and got["clamped"] == 0
        start = [0 if m < 0 else held[b] for b, m in enumerate(n)]
        for b, m in enumerate(n):
            if m > 0:
                k1, v1 = (x[b:b + 1, :, start[b]:start[b] + m].contiguous() for x in (K, V))
                s = _ints([start[b]])
                dq.dq_append_kv_paged(tab, k1, v1, s, kp, vp, table[b:b + 1], stats=stats)
                dq.dq_append_kv(tab, k1, v1, s, kc[b:b + 1], vc[b:b + 1], stats=stats)
            held[b] = start[b] + m if m >= 0 else 0
        assert lens.tolist() == held

    def attend(n_q):
        q = torch.randn(6, n_q, Hkv * G, 128, device="cuda")
        start = lens - n_q
        a, b = torch.empty_like(q), torch.empty_like(q)
        dq.dq_prefill_attention_window_paged(tab, q, kp, vp, table, start, window, sinks, a, stats=stats)
        dq.dq_prefill_attention_window(tab, q, kc, vc, start, window, sinks, b)
        assert torch.equal(a, b)
        if n_q == 1:
            dws = torch.empty(dq.dq_decode_workspace_bytes(tab, 6, Hkv * G, Hkv, 32 * mp), dtype=torch.uint8, device="cuda")
            x, y = q[:, 0].contiguous(), torch.empty_like(q[:, 0])
            z = torch.empty_like(y)
            dq.dq_decode_attention_window_paged(tab, x, kp, vp, table, lens, 32 * mp, window, sinks, y, dws, stats=stats)
            dq.dq_decode_attention_window(tab, x, kc, vc, lens, 32 * mp, window, sinks, z, dws)
            assert torch.equal(y, z)

    append([45, 45, 45, 0, 0, 0])  # prompts, chunk by chunk
    append([45, 45, 45, 0, 0, 0])
    append([45, 13, 45, 0, 0, 0])
    # Samples: rows 3 and 4 continue row 0, row 5 row 2; all write on from a shared prefix of their own.
    parent = [0, 1, 2, 0, 0, 2]
    pairs = torch.empty((6, 2), dtype=torch.int32, device="cuda")
    dq.dq_pages_fork(tab, refs, table, lens, _ints(parent), *spare, pairs, counts, ws)
    assert dq.page_counts_dict(counts)["pairs"] == 3 and dq.page_counts_dict(counts)["short_of"] == 0
    dq.dq_pages_copy(tab, kp, vp, pairs, counts, stats=stats)
    refs, table, lens = spare
    kc, vc = kc[parent].contiguous(), vc[parent].contiguous()
    held = [held[p] for p in parent]
    attend(13)
    for step in range(40):
        append([1] * 6)
        attend(1)
    append([-1, 1, -1, 1, 1, 1])
    # A compaction: the pages in use are the lowest ones afterwards.
    pairs = torch.empty((P // 2, 2), dtype=torch.int32, device="cuda")
    dq.dq_pages_compact(tab, refs, table, refs, table, pairs, counts, ws)
    dq.dq_pages_copy(tab, kp, vp, pairs, counts, stats=stats)
    c = dq.page_counts_dict(counts)
    live = P - c["free_pages"]
    assert c["pairs"] > 0 and bool((refs[:live] > 0).all()) and bool((refs[live:] == 0).all())
    kp[live:], vp[live:] = 0xFF, 0xFF
    attend(1)
    append([60, 1, 33, 1, 1, 1])  # new prompts take the rows that ended
    attend(1)
    append([-1] * 6)
    assert dq.page_counts_dict(counts)["free_pages"] == P and bool((refs == 0).all()) and bool((table == -1).all())
    s = dq.stats_dict(stats)
    assert s["bad_pages"] == s["integrity_errors"] == s["dropped_writes"] == s["wait_timeouts"] == 0
