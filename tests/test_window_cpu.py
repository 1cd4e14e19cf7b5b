"""Refusals of the windowed attention calls (no GPU): argument errors are
found on the host before any device work."""
import ctypes

import pytest
import torch

import decode_attention_dq_b200 as dq
from decode_attention_dq_b200 import _native as N

NULL, SHAPE, ALIGN = -1, -4, -6


def _decode(lib, window=8, sinks=0, scale=1.0, table=None, paged=False, num_pages=4, max_pages=4):
    if paged:
        return lib.dq_decode_attention_window_paged(None, None, 0, None, None, num_pages, table, max_pages, None, 1, 4, 1,
                                                    32, window, sinks, scale, None, 0, None, 0, None, None)
    return lib.dq_decode_attention_window(None, None, 0, None, None, None, 1, 4, 1, 32, 32, window, sinks, scale, None, 0,
                                          None, 0, None, None)


def _prefill(lib, window=8, sinks=0, scale=1.0, table=None, paged=False, num_pages=4, max_pages=4):
    if paged:
        return lib.dq_prefill_attention_window_paged(None, None, 0, None, None, num_pages, table, max_pages, None, 1, 2, 4,
                                                     1, window, sinks, scale, None, 0, None, 0, None, None)
    return lib.dq_prefill_attention_window(None, None, 0, None, None, None, 1, 2, 4, 1, 32, window, sinks, scale, None, 0,
                                           None, 0, None, None)


@pytest.mark.parametrize("call", [_decode, _prefill])
def test_window_arguments(call):
    lib = N.load()
    aligned, odd = ctypes.c_void_p(4096), ctypes.c_void_p(4097)
    for bad in (dict(window=0), dict(window=-3), dict(sinks=-1), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan"))):
        assert call(lib, **bad) == SHAPE, bad
        assert call(lib, paged=True, table=aligned, **bad) == SHAPE, bad
    assert call(lib) == NULL
    assert call(lib, paged=True) == NULL  # no page table
    assert call(lib, paged=True, table=odd) == ALIGN
    for bad in (dict(num_pages=0), dict(max_pages=0), dict(num_pages=2 ** 31 + 1), dict(max_pages=2 ** 40 + 1)):
        assert call(lib, paged=True, table=aligned, **bad) == SHAPE, bad


def test_workspace_of_nothing_is_zero():
    assert N.load().dq_prefill_window_workspace_bytes(None, 1, 1, 32, 1, 8, 0) == 0


def test_binding_refuses_tensors_that_are_not_on_a_gpu():
    q = torch.zeros(1, 4, 128)
    cache = torch.zeros(1, 1, 32, 36, dtype=torch.uint8)
    lens = torch.ones(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        dq.dq_decode_attention_window(None, q, cache, cache, lens, 32, 8, 0, q, cache)
    with pytest.raises(ValueError, match="CUDA"):
        dq.dq_prefill_attention_window(None, q[:, None], cache, cache, lens, 8, 0, q[:, None])


def test_binding_refuses_shapes_that_do_not_fit():
    N._check_int32("seq_lens", (torch.zeros(3, dtype=torch.int32), (3,)))
    for bad in (torch.zeros(2, dtype=torch.int32), torch.zeros(3, dtype=torch.int64), torch.zeros(3, 1, dtype=torch.int32)):
        with pytest.raises(ValueError, match="seq_lens"):
            N._check_int32("seq_lens", (bad, (3,)))
    q = torch.zeros(1, 4, 128)
    cache = torch.zeros(1, 1, 32, 36, dtype=torch.uint8)
    for args in ((torch.zeros(1, 4, 64), torch.zeros(1, 4, 64), cache, cache), (q, q[:, :2], cache, cache),
                 (q, q, cache.float(), cache), (q, q, cache, cache.int())):
        with pytest.raises(ValueError):
            N._check_heads(*args)
    with pytest.raises(ValueError, match="caches"):
        N._check_shapes("caches", cache, cache[:, :, :16], (1, 1, 32, 36), (1, 1, 32, 36))


@pytest.mark.parametrize("small", [torch.zeros(13, dtype=torch.int64), torch.zeros(14, dtype=torch.int32),
                                   torch.zeros(0, dtype=torch.int64)])
def test_binding_refuses_counters_without_room(small):
    with pytest.raises(ValueError, match="counters"):
        N._check_stats(small)
    with pytest.raises(ValueError, match="CUDA"):  # large enough, but not on a GPU
        N._check_stats(dq.new_stats(device="cpu"))
    N._check_stats(None)


@pytest.mark.parametrize("call", [_decode, _prefill])
def test_an_infinite_scale_is_refused(call):
    assert call(N.load(), scale=float("inf")) == SHAPE
    assert call(N.load(), paged=True, table=ctypes.c_void_p(4096), scale=float("inf")) == SHAPE
    assert call(N.load(), scale=3e38) == NULL
