"""Sliding-window attention with visible first tokens (dq_decode_attention_
window, dq_prefill_attention_window and their paged forms) against the fp64
definition over the oracle's dequantised cache.

Windows and first tokens that end inside a 32-token group and a 128-token
block, that meet, that cover everything or one token; lengths 0, 1 and around
a group's edge; ragged batches; every G; fp32 and bf16; 31-, 36- and 48-byte
containers; hidden tokens whose bytes are garbage and whose pages are gone;
replayed graphs and concurrent streams.
"""
import numpy as np
import pytest
import torch

import decode_attention_dq_b200 as dq
from decode_attention_dq_b200 import synth
from oracle import oracle as o
from tests import _common as cm
from tests import _window as W

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def _setup(B, Hkv, G, T, bits=2.26, v_levels=6):
    w = synth.scaled(synth.WORKLOADS["qwen3_8b_b16_t8k"], B=B, Hkv=Hkv, Hq=Hkv * G, T=T)
    K, V, _ = cm.inputs(w)
    lib, ref = cm.lib_tables(Hkv, bits, bits, v_levels=v_levels), cm.oracle_tables(Hkv, bits, bits, v_levels=v_levels)
    kc, vc = cm.gpu_append_all(lib, K, V, BF16)
    return w, lib, ref, kc, vc, cm.flat(kc), cm.flat(vc)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _workspace(lib, B, Hq, Hkv, T):
    return torch.empty(dq.dq_decode_workspace_bytes(lib, B, Hq, Hkv, T), dtype=torch.uint8, device="cuda")


def _decode(lib, q, kc, vc, lens, window, sinks, dtype=F32, stats=None, sm_scale=None):
    B, Hq, _ = q.shape
    qt = torch.from_numpy(q).to("cuda", dtype)
    out = torch.full(q.shape, float("nan"), dtype=dtype, device="cuda")
    ws = _workspace(lib, B, Hq, kc.shape[1], kc.shape[2])
    ws.fill_(0xFF)
    dq.dq_decode_attention_window(lib, qt, kc, vc, _ints(lens), kc.shape[2], window, sinks, out, ws, stats=stats,
                                  sm_scale=sm_scale)
    return out


def _rounded(q, dtype):
    return torch.from_numpy(q).to(dtype).float().numpy()


def _np(t):
    return t.float().cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 4), (32, 32), (33, 0), (64, 31), (100, 33), (250, 64),
                                          (257, 5), (1000, 3), (7, 1000)])
@pytest.mark.parametrize("times", [1, 11])  # one cluster per (b, h), and more rows than there are SMs
def test_decode_matches_definition(window, sinks, times):
    B, Hkv, G, T = 9 * times, 2, 4, 300
    w, lib, ref, kc, vc, rk, rv = _setup(B, Hkv, G, T)
    lens = [300, 0, 1, 31, 32, 33, 64, 97, 255] * times
    q = synth.q_block(w)
    stats = dq.new_stats()
    got = _np(_decode(lib, q, kc, vc, lens, window, sinks, stats=stats))
    want, bound = W.attention(ref, q[:, None], rk, rv, np.array(lens) - 1, window, sinks, chunk=False, half_levels=False)
    W.assert_within(got, want[:, 0], bound[:, 0], False, "window %d sinks %d" % (window, sinks))
    assert np.all(got[1] == 0.0)
    s = dq.stats_dict(stats)
    assert s["integrity_errors"] == 0 and s["clamped_lengths"] == 0


@pytest.mark.parametrize("G,bits,dtype", [(1, 1.96, F32), (2, 2.26, BF16), (8, 3.0, F32), (8, 2.26, BF16), (4, 3.0, BF16)])
@pytest.mark.parametrize("times", [1, 20])
def test_decode_group_sizes_and_types(G, bits, dtype, times):
    B, Hkv, T = 4 * times, 2, 500
    w, lib, ref, kc, vc, rk, rv = _setup(B, Hkv, G, T, bits)
    lens, window, sinks = [500, 411, 130, 17] * times, 129, 6
    q = _rounded(synth.q_block(w), dtype)
    got = _np(_decode(lib, q, kc, vc, lens, window, sinks, dtype=dtype))
    want, bound = W.attention(ref, q[:, None], rk, rv, np.array(lens) - 1, window, sinks, chunk=False,
                              half_levels=dtype == BF16)
    W.assert_within(got, want[:, 0], bound[:, 0], dtype == BF16, "G %d" % G)


@pytest.mark.parametrize("v_levels,bits", [(2, 2.26), (4, 1.96), (8, 1.96), (8, 2.26), (8, 3.0)])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("times", [1, 30])
def test_decode_value_tables_of_every_size(v_levels, bits, dtype, times):
    B, Hkv, G, T = 3 * times, 2, 2, 400
    w, lib, ref, kc, vc, rk, rv = _setup(B, Hkv, G, T, bits, v_levels)
    lens, q, stats = [400, 300, 90] * times, _rounded(synth.q_block(w), dtype), dq.new_stats()
    got = _np(_decode(lib, q, kc, vc, lens, 150, 5, dtype=dtype, stats=stats))
    want, bound = W.attention(ref, q[:, None], rk, rv, np.array(lens) - 1, 150, 5, chunk=False, half_levels=dtype == BF16)
    W.assert_within(got, want[:, 0], bound[:, 0], dtype == BF16, "%d levels" % v_levels)
    assert dq.stats_dict(stats)["integrity_errors"] == 0


@pytest.mark.parametrize("T", [1500, 3100, 6300])
def test_decode_long_windows(T):
    # One head: 47, 97 and 197 groups, i.e. 3 and 7 warps per CTA of a 16-CTA cluster, then the balanced split.
    w, lib, ref, kc, vc, rk, rv = _setup(1, 1, 4, T)
    q = synth.q_block(w)
    for window, sinks in ((T - 40, 7), (T // 2, 64)):
        got = _np(_decode(lib, q, kc, vc, [T], window, sinks))
        want, bound = W.attention(ref, q[:, None], rk, rv, [T - 1], window, sinks, chunk=False, half_levels=False)
        W.assert_within(got, want[:, 0], bound[:, 0], False, "T %d window %d" % (T, window))


def test_decode_many_sequences_and_a_scale():
    # More sequences than one pass of the prefix scan and lengths that leave rows empty.
    B, Hkv, G, T = 1500, 1, 1, 64
    w, lib, ref, kc, vc, rk, rv = _setup(B, Hkv, G, T)
    lens = [(b * 7) % 65 for b in range(B)]
    q = synth.q_block(w)
    got = _np(_decode(lib, q, kc, vc, lens, 20, 2, sm_scale=0.25))
    want, bound = W.attention(ref, q[:, None], rk, rv, np.array(lens) - 1, 20, 2, chunk=False, sm_scale=0.25, half_levels=False)
    W.assert_within(got, want[:, 0], bound[:, 0], False, "1500 sequences")


def test_decode_window_of_everything_is_the_call_without_one():
    B, Hkv, G, T = 3, 2, 4, 333
    w, lib, ref, kc, vc, rk, rv = _setup(B, Hkv, G, T)
    lens, q = [333, 100, 0], synth.q_block(w)
    qr = _rounded(q, BF16)
    half = cm.gpu_attention(lib, qr, kc, vc, lens, T_max=kc.shape[2], q_dtype=BF16, out_dtype=BF16)
    want, bound = W.attention(ref, q[:, None], rk, rv, np.array(lens) - 1, 333, 0, chunk=False, half_levels=False)
    for window, sinks in ((333, 0), (2 ** 40, 0), (1, 333), (200, 2 ** 40)):
        assert np.array_equal(_np(_decode(lib, qr, kc, vc, lens, window, sinks, dtype=BF16)), half)
        W.assert_within(_np(_decode(lib, q, kc, vc, lens, window, sinks)), want[:, 0], bound[:, 0], False, "everything")


def _pool_of(lib, cache, table, num_pages, keep):
    """A pool of garbage (0xFF: NaN norms) that holds the kept blocks of a cache where the table says."""
    B, Hkv, T_cap, C = cache.shape
    blocks = cache.reshape(B, Hkv, T_cap // 32, C, 32)
    pool = torch.full((num_pages, Hkv, C, 32), 0xFF, dtype=torch.uint8, device="cuda")
    for b in range(B):
        for j in range(T_cap // 32):
            if keep[b][j]:
                pool[int(table[b, j])] = blocks[b, :, j]
    return pool


def _paged(lib, kc, vc, lens, n_q, window, sinks, seed):
    """Pools and a table that hold only the blocks that some query sees."""
    B, nb = kc.shape[0], kc.shape[2] // 32
    num_pages = B * nb + 2
    table = torch.from_numpy(np.random.default_rng(seed).permutation(num_pages)[:B * nb].reshape(B, nb).astype(np.int32))
    keep = [[32 * j < L and (32 * j < sinks or 32 * j + 32 > L - n_q + 1 - window) for j in range(nb)] for L in lens]
    kp, vp = (_pool_of(lib, c, table, num_pages, keep) for c in (kc, vc))
    table[~torch.tensor(keep)] = -1
    return kp, vp, table.cuda()


@pytest.mark.parametrize("window,sinks", [(40, 0), (65, 5), (128, 64)])
@pytest.mark.parametrize("times", [1, 13])
def test_decode_paged_reads_only_what_is_visible(window, sinks, times):
    B, Hkv, G, T = 4 * times, 3, 2, 400
    w, lib, ref, kc, vc, _, _ = _setup(B, Hkv, G, T)
    lens, q = [400, 385, 66, 7] * times, synth.q_block(w)
    want = _decode(lib, q, kc, vc, lens, window, sinks)
    kp, vp, table = _paged(lib, kc, vc, lens, 1, window, sinks, 3)
    stats = dq.new_stats()
    out = torch.full(q.shape, float("nan"), device="cuda")
    dq.dq_decode_attention_window_paged(lib, torch.from_numpy(q).cuda(), kp, vp, table, _ints(lens), 400, window, sinks,
                                        out, _workspace(lib, B, Hkv * G, Hkv, 400), stats=stats)
    assert torch.equal(out, want)
    s = dq.stats_dict(stats)
    assert s["bad_pages"] == 0 and s["integrity_errors"] == 0


@pytest.mark.parametrize("times", [1, 40])
def test_decode_hidden_and_later_tokens_may_be_garbage(times):
    B, Hkv, G, T = 2 * times, 2, 4, 320
    w, lib, ref, kc, vc, _, _ = _setup(B, Hkv, G, T)
    lens, window, sinks, q = [290, 155] * times, 70, 3, synth.q_block(w)
    want = _decode(lib, q, kc, vc, lens, window, sinks)
    for c in (kc, vc):
        blocks = c.reshape(B, Hkv, T // 32, c.shape[3], 32)
        for b, L in enumerate(lens):
            for t in range(T):
                if not (t < L and (t < sinks or t >= L - window)):
                    blocks[b, :, t // 32, :, t % 32] = 0xFF
    stats = dq.new_stats()
    assert torch.equal(_decode(lib, q, kc, vc, lens, window, sinks, stats=stats), want)
    assert dq.stats_dict(stats)["integrity_errors"] == 0


@pytest.mark.parametrize("rows", [2, 160])
def test_decode_counts_visible_corrupt_containers_and_long_lengths(rows):
    B, Hkv, G, T = rows, 1, 2, 96
    w, lib, ref, kc, vc, _, _ = _setup(B, Hkv, G, T)
    q = synth.q_block(w)
    rest = [50] * (rows - 2)
    want = _decode(lib, q, kc, vc, [96, 96] + rest, 30, 2)
    for t in (95, 40, 1):  # two visible ones, one hidden
        vc.reshape(B, Hkv, 3, 36, 32)[0, :, t // 32, 0:2, t % 32] = 0xFF
    stats = dq.new_stats()
    got = _decode(lib, q, kc, vc, [2000, -5] + rest, 30, 2, stats=stats)
    assert torch.isfinite(got).all() and torch.all(got[1] == 0)
    s = dq.stats_dict(stats)
    assert s["integrity_errors"] == 2 and s["clamped_lengths"] == 2
    assert torch.equal(_decode(lib, q, kc, vc, [96, 96] + rest, 30, 2)[1:], want[1:])


def _prefill(lib, q, kc, vc, start, window, sinks, q_dtype=F32, out_dtype=F32, stats=None, workspace=None):
    qt = torch.from_numpy(q).to("cuda", q_dtype)
    out = torch.full(q.shape, float("nan"), dtype=out_dtype, device="cuda")
    dq.dq_prefill_attention_window(lib, qt, kc, vc, _ints(start), window, sinks, out, stats=stats, workspace=workspace)
    return out


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 130), (31, 4), (40, 0), (128, 128), (129, 1), (200, 33), (300, 5),
                                          (5000, 0), (3, 5000)])
def test_prefill_matches_definition(window, sinks):
    B, Hkv, G, T = 3, 2, 4, 700
    w, lib, ref, kc, vc, rk, rv = _setup(B, Hkv, G, T)
    n_q, start = 150, [550, 0, 333]
    q = synth.q_chunk(w, n_q)
    stats = dq.new_stats()
    got = _np(_prefill(lib, q, kc, vc, start, window, sinks, stats=stats))
    want, bound = W.attention(ref, q, rk, rv, start, window, sinks, chunk=True)
    W.assert_within(got, want, bound, False, "window %d sinks %d" % (window, sinks))
    s = dq.stats_dict(stats)
    assert s["wait_timeouts"] == 0 and s["integrity_errors"] == 0 and s["clamped_lengths"] == 0


@pytest.mark.parametrize("G,bits,q_dtype,out_dtype", [(1, 1.96, F32, BF16), (2, 2.26, BF16, BF16), (8, 3.0, BF16, F32),
                                                      (8, 2.26, F32, F32)])
def test_prefill_group_sizes_and_types(G, bits, q_dtype, out_dtype):
    B, Hkv, T = 2, 2, 600
    w, lib, ref, kc, vc, rk, rv = _setup(B, Hkv, G, T, bits)
    n_q, start, window, sinks = 141, [459, 201], 133, 7
    q = _rounded(synth.q_chunk(w, n_q), q_dtype)
    got = _np(_prefill(lib, q, kc, vc, start, window, sinks, q_dtype, out_dtype))
    want, bound = W.attention(ref, q, rk, rv, start, window, sinks, chunk=True, half_weights=out_dtype == BF16)
    W.assert_within(got, want, bound, out_dtype == BF16, "G %d" % G)


def test_prefill_bf16_outputs_in_windows_long_and_short():
    # One fp16 value per weight: many small weights, one large one, sinks far behind.
    B, Hkv, G, T = 2, 2, 4, 900
    w, lib, ref, kc, vc, rk, rv = _setup(B, Hkv, G, T)
    n_q, start = 130, [770, 300]
    q = _rounded(synth.q_chunk(w, n_q), BF16)
    for window, sinks, scale in ((1, 0, 1.0), (800, 0, 1.0), (64, 200, 0.01), (500, 3, 4.0)):
        got = _np(_prefill(lib, q * np.float32(scale), kc, vc, start, window, sinks, F32, BF16))
        want, bound = W.attention(ref, q * np.float32(scale), rk, rv, start, window, sinks, chunk=True, half_weights=True)
        W.assert_within(got, want, bound, True, "window %d scale %g" % (window, scale))


def test_prefill_rows_outside_the_cache():
    B, Hkv, G, T = 5, 1, 2, 416
    w, lib, ref, kc, vc, rk, rv = _setup(B, Hkv, G, T)
    n_q, start, window, sinks = 70, [-4, T - 3, 40, T + 5, -1000], 50, 3
    q = synth.q_chunk(w, n_q)
    stats = dq.new_stats()
    got = _np(_prefill(lib, q, kc, vc, start, window, sinks, stats=stats))
    want, bound = W.attention(ref, q, rk, rv, start, window, sinks, chunk=True)
    W.assert_within(got, want, bound, False, "rows outside")
    s = dq.stats_dict(stats)
    assert s["clamped_lengths"] == (4 + 67 + 70 + 70) * G and s["wait_timeouts"] == 0


def test_prefill_window_of_everything_is_the_call_without_one():
    B, Hkv, G, T = 2, 2, 4, 300
    w, lib, ref, kc, vc, _, _ = _setup(B, Hkv, G, T)
    n_q, start = 60, [240, 17]
    q = synth.q_chunk(w, n_q)
    full = torch.full(q.shape, float("nan"), device="cuda")
    dq.dq_prefill_attention(lib, torch.from_numpy(q).cuda(), kc, vc, _ints(start), full)
    for window, sinks in ((320, 0), (2 ** 40, 1), (1, 320)):
        assert torch.equal(_prefill(lib, q, kc, vc, start, window, sinks), full)


def test_prefill_chunks_of_one_token_are_decode_steps():
    B, Hkv, G, T = 3, 2, 4, 500
    w, lib, ref, kc, vc, rk, rv = _setup(B, Hkv, G, T)
    lens, window, sinks = [500, 37, 260], 99, 4
    q = synth.q_block(w)
    got = _np(_prefill(lib, q[:, None].copy(), kc, vc, np.array(lens) - 1, window, sinks))[:, 0]
    want, bound = W.attention(ref, q[:, None], rk, rv, np.array(lens) - 1, window, sinks, chunk=True)
    W.assert_within(got, want[:, 0], bound[:, 0], False, "chunk of one")
    W.assert_within(_np(_decode(lib, q, kc, vc, lens, window, sinks)), want[:, 0], bound[:, 0], False, "decode")


@pytest.mark.parametrize("window,sinks", [(64, 0), (200, 40), (33, 300)])
def test_prefill_paged_reads_only_what_is_visible(window, sinks):
    B, Hkv, G, T = 2, 2, 4, 1056
    w, lib, ref, kc, vc, _, _ = _setup(B, Hkv, G, T)
    n_q, lens = 90, [1050, 700]
    start = [L - n_q for L in lens]
    q = synth.q_chunk(w, n_q)
    want = _prefill(lib, q, kc, vc, start, window, sinks)
    kp, vp, table = _paged(lib, kc, vc, lens, n_q, window, sinks, 5)
    stats = dq.new_stats()
    out = torch.full(q.shape, float("nan"), device="cuda")
    dq.dq_prefill_attention_window_paged(lib, torch.from_numpy(q).cuda(), kp, vp, table, _ints(start), window, sinks, out,
                                         stats=stats)
    assert torch.equal(out, want)
    s = dq.stats_dict(stats)
    assert s["bad_pages"] == 0 and s["integrity_errors"] == 0 and s["wait_timeouts"] == 0


def test_prefill_corrupt_norms_stay_with_the_rows_that_see_them():
    # Token 60's value has a NaN norm: the queries whose window has left it behind do not see it.
    B, Hkv, G, T = 1, 1, 4, 256
    w, lib, ref, kc, vc, _, _ = _setup(B, Hkv, G, T)
    n_q, start, window = 128, [50], 20
    q = synth.q_chunk(w, n_q)
    want = _np(_prefill(lib, q, kc, vc, start, window, 0))
    vc.reshape(1, 1, 8, 36, 32)[0, :, 1, 0:2, 28] = 0xFF
    stats = dq.new_stats()
    got = _np(_prefill(lib, q, kc, vc, start, window, 0, stats=stats))
    pos = 50 + np.arange(n_q)
    blind = (pos < 60) | (pos - window >= 60)
    assert np.array_equal(got[0, blind], want[0, blind]) and np.all(np.isfinite(got))
    assert dq.stats_dict(stats)["integrity_errors"] == 1


def test_prefill_in_waves_is_bit_identical():
    B, Hkv, G, T = 2, 3, 2, 500
    w, lib, ref, kc, vc, _, _ = _setup(B, Hkv, G, T)
    n_q, start, window, sinks = 77, [423, 100], 150, 9
    q = synth.q_chunk(w, n_q)
    want = _prefill(lib, q, kc, vc, start, window, sinks)
    row = dq.dq_prefill_window_workspace_bytes(lib, 1, 1, kc.shape[2], n_q, window, sinks)
    # One 128-token block of first tokens, at most three that 226 consecutive
    # tokens meet, however long the cache.
    assert row == dq.dq_prefill_window_workspace_bytes(lib, 1, 1, 2 ** 20, n_q, window, sinks)
    assert row == 4 * dq.dq_prefill_workspace_bytes(lib, 1, 1, 128)
    for rows in (1, 4):
        ws = torch.full((rows * row,), 0xFF, dtype=torch.uint8, device="cuda")
        assert torch.equal(_prefill(lib, q, kc, vc, start, window, sinks, workspace=ws), want)
    with pytest.raises(dq.DqError, match="workspace"):
        _prefill(lib, q, kc, vc, start, window, sinks, workspace=torch.empty(row - 16, dtype=torch.uint8, device="cuda"))


def test_offsets_past_four_gigabytes():
    # 2^27 tokens, 4.8 GB per stream: the first 5 and the last 100 are there, the rest is garbage.
    B, Hkv, G, T, far = 1, 1, 4, 105, 2 ** 27
    w, lib, ref, kc, vc, rk, rv = _setup(B, Hkv, G, T)
    K, V, _ = cm.inputs(w)
    big = [torch.full((1, 1, far, 36), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(2)]
    for part, at in ((slice(0, 5), 0), (slice(5, 105), far - 100)):
        k, v = (torch.from_numpy(x[:, :, part]).cuda().bfloat16().contiguous() for x in (K, V))
        dq.dq_append_kv(lib, k, v, _ints([at]), *big)
    q = synth.q_block(w)
    want, bound = W.attention(ref, q[:, None], rk, rv, [T - 1], T, 0, chunk=False, half_levels=False)
    stats = dq.new_stats()
    W.assert_within(_np(_decode(lib, q, *big, [far], 100, 5, stats=stats)), want[:, 0], bound[:, 0], False, "decode")
    # The same 60 tokens and first 5 for every query of a chunk, wherever they are.
    qc = synth.q_chunk(w, 40)
    want, bound = W.attention(ref, qc, rk, rv, [T - 40], 60, 5, chunk=True)
    W.assert_within(_np(_prefill(lib, qc, *big, [far - 40], 60, 5, stats=stats)), want, bound, False, "chunk")
    s = dq.stats_dict(stats)
    assert s["wait_timeouts"] == 0 and s["clamped_lengths"] == 0 and s["integrity_errors"] == 0


def test_tiny_queries_and_scales_stay_finite():
    # Logits far below one step: the weights are equal, masked tokens weigh nothing.
    B, Hkv, G, T = 1, 1, 4, 200
    w, lib, ref, kc, vc, rk, rv = _setup(B, Hkv, G, T)
    n_q, start, window = 40, [150], 25
    q = synth.q_chunk(w, n_q)
    want, bound = W.attention(ref, 0 * q, rk, rv, start, window, 2, chunk=True)
    for qs in (np.float32(1e-38) * q, 0 * q):
        W.assert_within(_np(_prefill(lib, qs, kc, vc, start, window, 2)), want, bound + 1e-6, False, "tiny queries")
    out = torch.empty(q.shape, device="cuda")
    dq.dq_prefill_attention_window(lib, torch.from_numpy(q).cuda(), kc, vc, _ints(start), window, 2, out, sm_scale=1e-37)
    W.assert_within(_np(out), want, bound + 1e-6, False, "tiny scale")


def test_captured_decode_follows_the_lengths():
    B, Hkv, G, T = 2, 2, 4, 256
    w, lib, ref, kc, vc, _, _ = _setup(B, Hkv, G, T)
    qt, seq = torch.from_numpy(synth.q_block(w)).cuda(), _ints([200, 50])
    out, ws = torch.empty_like(qt), _workspace(lib, B, Hkv * G, Hkv, T)
    call = lambda: dq.dq_decode_attention_window(lib, qt, kc, vc, seq, T, 60, 3, out, ws)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for lens in ([256, 1], [77, 230]):
        seq.copy_(_ints(lens))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, _decode(lib, synth.q_block(w), kc, vc, lens, 60, 3))


def test_two_streams_with_their_own_workspaces():
    B, Hkv, G, T = 2, 2, 4, 512
    w, lib, ref, kc, vc, _, _ = _setup(B, Hkv, G, T)
    n_q, q1, qc = 64, synth.q_block(w), synth.q_chunk(w, 64)
    a, b = _decode(lib, q1, kc, vc, [512, 300], 100, 4), _prefill(lib, qc, kc, vc, [448, 100], 100, 4)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(10):
        with torch.cuda.stream(s1):
            x = _decode(lib, q1, kc, vc, [512, 300], 100, 4)
        with torch.cuda.stream(s2):
            y = _prefill(lib, qc, kc, vc, [448, 100], 100, 4)
        torch.cuda.synchronize()
        assert torch.equal(x, a) and torch.equal(y, b)
