"""ctypes binding of libdq (include/dq.h): the same entry points, argument
marshalling only. PyTorch supplies device memory and streams; every step of
the path runs in libdq's CUDA kernels. There is no CPU fallback: if libdq.so
is missing, loading raises.
"""
from __future__ import annotations

import ctypes as C
import os
from dataclasses import dataclass

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
# DQ_LIBRARY selects another build of the same ABI (lib/libdq_checked.so:
# the attention kernels also count containers decoded past their bytes).
LIB_PATH = os.environ.get("DQ_LIBRARY") or os.path.join(HERE, "lib", "libdq.so")

DQ_OK = 0
DQ_F32, DQ_BF16 = 0, 1
DQ_STREAM_K, DQ_STREAM_V = 0, 1
STATS_FIELDS = ("k_syms_drifted", "v_syms_drifted", "k_cont_drifted", "v_cont_drifted",
                "overflow_fallbacks", "integrity_errors", "nonfinite_inputs",
                "dropped_writes", "clamped_lengths", "bad_pages", "wait_timeouts",
                "k_syms_filled", "v_syms_filled", "overreads")
EXPORTED = ("dq_config_default", "dq_build_tables", "dq_free_tables", "dq_get_stream_table",
            "dq_get_stream_design", "dq_get_signs", "dq_append_kv", "dq_decode_workspace_bytes",
            "dq_decode_attention", "dq_decode_symbols", "dq_error_string", "dq_last_cuda_error",
            "dq_design_stream", "dq_decode_attention_noalloc", "dq_append_workspace_bytes",
            "dq_append_kv_ws", "dq_append_kv_paged", "dq_decode_attention_paged",
            "dq_prefill_attention", "dq_prefill_attention_paged", "dq_prefill_workspace_bytes",
            "dq_decode_attention_window", "dq_decode_attention_window_paged", "dq_prefill_attention_window",
            "dq_prefill_attention_window_paged", "dq_prefill_window_workspace_bytes",
            "dq_pages_workspace_bytes", "dq_pages_advance", "dq_pages_fork", "dq_pages_compact", "dq_pages_copy")
PAGE_COUNT_FIELDS = ("free_pages", "taken", "released", "short_of", "bad", "clamped", "pairs", "reserved")


class DqConfig(C.Structure):
    _fields_ = [
        ("head_dim", C.c_int32), ("k_levels", C.c_int32), ("v_levels", C.c_int32),
        ("prob_bits", C.c_int32), ("k_container_bytes", C.c_int32),
        ("v_container_bytes", C.c_int32), ("k_bits_per_value", C.c_float),
        ("v_bits_per_value", C.c_float), ("n_kv_heads", C.c_int32), ("drift_mode", C.c_int32),
        ("sign_seed", C.c_uint64), ("k_rate_offset", C.c_float), ("v_rate_offset", C.c_float),
    ]


class DqError(RuntimeError):
    def __init__(self, fn, code):
        lib = load()
        msg = lib.dq_error_string(code).decode()
        if code == -8:
            msg += " (cuda error %d)" % lib.dq_last_cuda_error()
        super().__init__("%s failed: %s [%d]" % (fn, msg, code))
        self.code = code


_lib = None


def load():
    """Load libdq.so; raises if it has not been built (no fallback)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError("libdq.so not built at %s; run `python -m decode_attention_dq_b200.build`"
                          % LIB_PATH)
    lib = C.CDLL(LIB_PATH)
    vp, i32, i64, P = C.c_void_p, C.c_int32, C.c_int64, C.POINTER
    lib.dq_config_default.argtypes = [P(DqConfig)]
    lib.dq_config_default.restype = None
    lib.dq_build_tables.argtypes = [P(DqConfig), P(vp)]
    lib.dq_free_tables.argtypes = [vp]
    lib.dq_free_tables.restype = None
    lib.dq_get_stream_table.argtypes = [vp, C.c_int, vp, vp, vp, vp, vp, vp, vp]
    lib.dq_get_stream_design.argtypes = [vp, C.c_int, vp, vp, vp, vp, vp]
    lib.dq_get_signs.argtypes = [vp, vp]
    lib.dq_append_kv.argtypes = [vp, vp, vp, C.c_int, C.c_int, C.c_int, C.c_int, vp, vp, vp,
                                 i64, vp, vp]
    lib.dq_append_workspace_bytes.argtypes = [vp, C.c_int, C.c_int, C.c_int]
    lib.dq_append_workspace_bytes.restype = C.c_size_t
    lib.dq_append_kv_ws.argtypes = [vp, vp, vp, C.c_int, C.c_int, C.c_int, C.c_int, vp, vp, vp,
                                    i64, vp, C.c_size_t, vp, vp]
    lib.dq_append_kv_paged.argtypes = [vp, vp, vp, C.c_int, C.c_int, C.c_int, C.c_int, vp, vp, vp,
                                       i64, vp, i64, vp, C.c_size_t, vp, vp]
    lib.dq_decode_attention_paged.argtypes = [vp, vp, C.c_int, vp, vp, i64, vp, i64, vp, C.c_int,
                                              C.c_int, C.c_int, i64, C.c_float, vp, C.c_int, vp,
                                              C.c_size_t, vp, vp]
    lib.dq_decode_workspace_bytes.argtypes = [vp, C.c_int, C.c_int, C.c_int, i64]
    lib.dq_decode_workspace_bytes.restype = C.c_size_t
    lib.dq_decode_attention.argtypes = [vp, vp, C.c_int, vp, vp, vp, C.c_int, C.c_int, C.c_int,
                                        i64, i64, C.c_float, vp, C.c_int, vp, C.c_size_t, vp, vp]
    lib.dq_decode_symbols.argtypes = [vp, vp, C.c_int, i64, vp, vp, vp, vp, vp]
    lib.dq_decode_attention_noalloc.argtypes = [vp, vp, C.c_int, vp, vp, vp, C.c_int, C.c_int,
                                                C.c_int, i64, i64, C.c_float, vp, C.c_int, vp, vp]
    lib.dq_prefill_workspace_bytes.argtypes = [vp, C.c_int, C.c_int, i64]
    lib.dq_prefill_workspace_bytes.restype = C.c_size_t
    lib.dq_prefill_attention.argtypes = [vp, vp, C.c_int, vp, vp, vp, C.c_int, C.c_int, C.c_int,
                                         C.c_int, i64, C.c_float, vp, C.c_int, vp, C.c_size_t, vp, vp]
    lib.dq_prefill_attention_paged.argtypes = [vp, vp, C.c_int, vp, vp, i64, vp, i64, vp, C.c_int,
                                               C.c_int, C.c_int, C.c_int, C.c_float, vp, C.c_int, vp,
                                               C.c_size_t, vp, vp]
    lib.dq_decode_attention_window.argtypes = [vp, vp, C.c_int, vp, vp, vp, C.c_int, C.c_int, C.c_int, i64, i64,
                                               i64, i64, C.c_float, vp, C.c_int, vp, C.c_size_t, vp, vp]
    lib.dq_decode_attention_window_paged.argtypes = [vp, vp, C.c_int, vp, vp, i64, vp, i64, vp, C.c_int, C.c_int,
                                                     C.c_int, i64, i64, i64, C.c_float, vp, C.c_int, vp, C.c_size_t,
                                                     vp, vp]
    lib.dq_prefill_window_workspace_bytes.argtypes = [vp, C.c_int, C.c_int, i64, C.c_int, i64, i64]
    lib.dq_prefill_window_workspace_bytes.restype = C.c_size_t
    lib.dq_prefill_attention_window.argtypes = [vp, vp, C.c_int, vp, vp, vp, C.c_int, C.c_int, C.c_int, C.c_int, i64,
                                                i64, i64, C.c_float, vp, C.c_int, vp, C.c_size_t, vp, vp]
    lib.dq_prefill_attention_window_paged.argtypes = [vp, vp, C.c_int, vp, vp, i64, vp, i64, vp, C.c_int, C.c_int,
                                                      C.c_int, C.c_int, i64, i64, C.c_float, vp, C.c_int, vp,
                                                      C.c_size_t, vp, vp]
    lib.dq_pages_workspace_bytes.argtypes = [vp, i64, C.c_int, i64]
    lib.dq_pages_workspace_bytes.restype = C.c_size_t
    lib.dq_pages_advance.argtypes = [vp, i64, vp, vp, i64, vp, vp, C.c_int, i64, i64, vp, vp, vp, vp, vp, C.c_size_t, vp]
    lib.dq_pages_fork.argtypes = [vp, i64, vp, vp, i64, vp, C.c_int, vp, C.c_int, vp, vp, vp, vp, vp, vp, C.c_size_t, vp]
    lib.dq_pages_compact.argtypes = [vp, i64, vp, vp, i64, C.c_int, vp, vp, vp, vp, vp, C.c_size_t, vp]
    lib.dq_pages_copy.argtypes = [vp, vp, vp, i64, i64, i64, i64, vp, i64, vp, vp, vp]
    lib.dq_error_string.argtypes = [C.c_int]
    lib.dq_error_string.restype = C.c_char_p
    lib.dq_last_cuda_error.argtypes = []
    lib.dq_design_stream.argtypes = [i32, i32, C.c_double, vp, vp, vp, vp, vp, vp, vp, vp]
    _lib = lib
    return lib


def _check(fn, code):
    if code != DQ_OK:
        raise DqError(fn, code)


def _ptr(t):
    return C.c_void_p(t.data_ptr()) if t is not None else None


def _addr(t):
    return t.data_ptr() if t is not None else None


def _stream(stream):
    if stream is None:  # (the current stream's handle without building a Stream object: 0.3 us instead of 3)
        return C.c_void_p(torch._C._cuda_getCurrentRawStream(torch.cuda.current_device()))
    return C.c_void_p(stream.cuda_stream)


def _workspace_for(nbytes: int, device, stream) -> torch.Tensor:
    """A workspace that lives for one call, from the pool of the stream that
    the call runs on: a block of another stream's pool may still be in use by
    work queued there, and may be handed to such work before the call has run."""
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return DQ_F32
    if t.dtype == torch.bfloat16:
        return DQ_BF16
    raise TypeError("dtype must be float32 or bfloat16, got %s" % t.dtype)


def dq_config_default(**overrides) -> DqConfig:
    cfg = DqConfig()
    load().dq_config_default(C.byref(cfg))
    for k, v in overrides.items():
        setattr(cfg, k, v)
    return cfg


@dataclass
class StreamTable:
    n_levels: int
    container_bytes: int
    levels: list
    thresholds: list
    freq: list
    cum: list
    cost: list


class Tables:
    """Owns a dq_tables handle (built on the current CUDA device)."""

    def __init__(self, cfg: DqConfig):
        self._h = C.c_void_p()
        _check("dq_build_tables", load().dq_build_tables(C.byref(cfg), C.byref(self._h)))
        self.cfg = cfg
        self.n_kv_heads = cfg.n_kv_heads
        self.k = self.stream_table(DQ_STREAM_K)
        self.v = self.stream_table(DQ_STREAM_V)

    @property
    def handle(self):
        return self._h

    def stream_table(self, kind: int) -> StreamTable:
        n = C.c_int32(); cb = C.c_int32()
        lev = (C.c_float * 8)(); thr = (C.c_float * 7)(); f = (C.c_uint32 * 8)()
        cum = (C.c_uint32 * 9)(); cost = (C.c_float * 8)()
        _check("dq_get_stream_table", load().dq_get_stream_table(
            self._h, kind, C.byref(n), C.byref(cb), lev, thr, f, cum, cost))
        nl = n.value
        return StreamTable(nl, cb.value, list(lev)[:nl], list(thr)[:nl - 1], list(f)[:nl],
                           list(cum)[:nl + 1], list(cost)[:nl])

    def design(self, kind: int) -> dict:
        lam = C.c_double(); ent = C.c_double(); rate = C.c_double(); mse = C.c_double()
        lm = C.c_int32()
        _check("dq_get_stream_design", load().dq_get_stream_design(
            self._h, kind, C.byref(lam), C.byref(ent), C.byref(rate), C.byref(mse), C.byref(lm)))
        return dict(lam=lam.value, entropy=ent.value, rate=rate.value, mse=mse.value,
                    is_lloyd_max=bool(lm.value))

    def signs(self):
        buf = (C.c_int8 * (self.n_kv_heads * 128))()
        _check("dq_get_signs", load().dq_get_signs(self._h, buf))
        return torch.tensor(list(buf), dtype=torch.int8).reshape(self.n_kv_heads, 128)

    def close(self):
        if self._h:
            load().dq_free_tables(self._h)
            self._h = C.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def dq_build_tables(cfg: DqConfig | None = None, **overrides) -> Tables:
    if cfg is None:
        cfg = dq_config_default(**overrides)
    return Tables(cfg)


def new_stats(device=None) -> torch.Tensor:
    """A zeroed device dq_stats (one uint64 per field of STATS_FIELDS)."""
    return torch.zeros(len(STATS_FIELDS), dtype=torch.int64, device=device or "cuda")


def stats_dict(stats: torch.Tensor) -> dict:
    vals = stats.cpu().tolist()
    return dict(zip(STATS_FIELDS, vals))


def new_cache(B: int, Hkv: int, T_cap: int, C: int, device=None) -> torch.Tensor:
    """Zeroed uint8 cache of shape [B, Hkv, T_cap, C] (T_cap a multiple of 32).
    The bytes are in the library's interleaved layout; use containers_of()
    to read flat containers."""
    assert T_cap % 32 == 0, "T_cap must be a multiple of 32"
    return torch.zeros((B, Hkv, T_cap, C), dtype=torch.uint8, device=device or "cuda")


def containers_of(cache: torch.Tensor) -> torch.Tensor:
    """Flat containers [B, Hkv, T_cap, C] (a copy) of a cache whose bytes are in
    the interleaved layout [B][Hkv][T_cap/32][C][32]."""
    B, H, T_cap, C = cache.shape
    return cache.reshape(B, H, T_cap // 32, C, 32).transpose(-1, -2).reshape(B, H, T_cap, C).contiguous()


def dq_append_workspace_bytes(tab: Tables, B: int, Hkv: int, n_new: int) -> int:
    return int(load().dq_append_workspace_bytes(tab.handle, B, Hkv, n_new))


def dq_append_kv(tab: Tables, k: torch.Tensor, v: torch.Tensor, start_pos: torch.Tensor,
                 kcache: torch.Tensor, vcache: torch.Tensor, stats: torch.Tensor | None = None,
                 stream=None, workspace: torch.Tensor | None = None) -> None:
    """k, v: [B, Hkv, n_new, 128] (f32/bf16, contiguous, CUDA); start_pos int32 [B];
    caches uint8 [B, Hkv, T_cap, C] holding the interleaved layout (see new_cache).
    Calls dq_append_kv_ws; without `workspace` one is taken from PyTorch's
    allocator on the caches' device. workspace=False calls dq_append_kv (drift
    inside the encode kernel)."""
    B, Hkv, n_new, d = k.shape
    assert d == 128 and v.shape == k.shape and k.dtype == v.dtype
    assert k.is_contiguous() and v.is_contiguous() and kcache.is_contiguous() and vcache.is_contiguous()
    assert start_pos.dtype == torch.int32 and kcache.dtype == torch.uint8
    T_cap = kcache.shape[2]
    if workspace is False:
        _check("dq_append_kv", load().dq_append_kv(
            tab.handle, _ptr(k), _ptr(v), _dtype_code(k), B, Hkv, n_new, _ptr(start_pos),
            _ptr(kcache), _ptr(vcache), T_cap, _ptr(stats), _stream(stream)))
        return
    if workspace is None:
        nbytes = dq_append_workspace_bytes(tab, B, Hkv, n_new)
        workspace = _workspace_for(max(nbytes, 16), kcache.device, stream)
    _check("dq_append_kv_ws", load().dq_append_kv_ws(
        tab.handle, _ptr(k), _ptr(v), _dtype_code(k), B, Hkv, n_new, _ptr(start_pos),
        _ptr(kcache), _ptr(vcache), T_cap, _ptr(workspace), workspace.numel(), _ptr(stats),
        _stream(stream)))


def dq_decode_workspace_bytes(tab: Tables, B: int, Hq: int, Hkv: int, T_max: int) -> int:
    return int(load().dq_decode_workspace_bytes(tab.handle, B, Hq, Hkv, T_max))


def dq_decode_attention(tab: Tables, q: torch.Tensor, kcache: torch.Tensor, vcache: torch.Tensor,
                        seq_lens: torch.Tensor, T_max: int, out: torch.Tensor,
                        workspace: torch.Tensor, sm_scale: float | None = None,
                        stats: torch.Tensor | None = None, stream=None) -> None:
    """q [B, Hq, 128]; caches uint8 [B, Hkv, T_cap, C]; seq_lens int32 [B];
    out [B, Hq, 128] (f32/bf16); workspace uint8 with dq_decode_workspace_bytes."""
    B, Hq, d = q.shape
    Hkv, T_cap = kcache.shape[1], kcache.shape[2]
    assert d == 128 and q.is_contiguous() and out.is_contiguous() and seq_lens.dtype == torch.int32
    if sm_scale is None:
        sm_scale = 128 ** -0.5
    _check("dq_decode_attention", load().dq_decode_attention(
        tab.handle, _ptr(q), _dtype_code(q), _ptr(kcache), _ptr(vcache), _ptr(seq_lens), B, Hq,
        Hkv, T_cap, T_max, float(sm_scale), _ptr(out), _dtype_code(out), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(stats), _stream(stream)))


def dq_decode_attention_noalloc(tab: Tables, q: torch.Tensor, kcache: torch.Tensor,
                                vcache: torch.Tensor, seq_lens: torch.Tensor, T_max: int,
                                out: torch.Tensor, sm_scale: float | None = None,
                                stats: torch.Tensor | None = None, stream=None) -> None:
    """dq_decode_attention for callers that cannot allocate: no workspace
    argument; the library's fixed 8 MiB device scratch array is used instead
    (shared by all calls on a device, so overlapping calls must be ordered)."""
    B, Hq, d = q.shape
    Hkv, T_cap = kcache.shape[1], kcache.shape[2]
    assert d == 128 and q.is_contiguous() and out.is_contiguous() and seq_lens.dtype == torch.int32
    if sm_scale is None:
        sm_scale = 128 ** -0.5
    _check("dq_decode_attention_noalloc", load().dq_decode_attention_noalloc(
        tab.handle, _ptr(q), _dtype_code(q), _ptr(kcache), _ptr(vcache), _ptr(seq_lens), B, Hq,
        Hkv, T_cap, T_max, float(sm_scale), _ptr(out), _dtype_code(out), _ptr(stats),
        _stream(stream)))


def dq_prefill_workspace_bytes(tab: Tables, B: int, Hkv: int, T_cap: int) -> int:
    """Bytes of the dq_prefill_attention workspace (decoded tiles)."""
    return int(load().dq_prefill_workspace_bytes(tab.handle, B, Hkv, T_cap))


def _prefill_ws(tab, workspace, B, Hkv, T_cap, device, stream):
    if workspace is None:
        workspace = _workspace_for(dq_prefill_workspace_bytes(tab, B, Hkv, T_cap), device, stream)
    return workspace


def dq_prefill_attention(tab: Tables, q: torch.Tensor, kcache: torch.Tensor, vcache: torch.Tensor,
                         q_start: torch.Tensor, out: torch.Tensor, workspace: torch.Tensor | None = None,
                         sm_scale: float | None = None, stats: torch.Tensor | None = None,
                         stream=None) -> None:
    """Chunked-prefill attention: q [B, n_q, Hq, 128] (query token i of
    sequence b at position q_start[b] + i, causal over the cache); caches
    uint8 [B, Hkv, T_cap, C]; q_start int32 [B]; out [B, n_q, Hq, 128];
    workspace uint8 of dq_prefill_workspace_bytes (allocated if None)."""
    B, n_q, Hq, d = q.shape
    Hkv, T_cap = kcache.shape[1], kcache.shape[2]
    assert d == 128 and q.is_contiguous() and out.is_contiguous() and q_start.dtype == torch.int32
    assert out.shape == q.shape
    if sm_scale is None:
        sm_scale = 128 ** -0.5
    workspace = _prefill_ws(tab, workspace, B, Hkv, T_cap, q.device, stream)
    _check("dq_prefill_attention", load().dq_prefill_attention(
        tab.handle, _ptr(q), _dtype_code(q), _ptr(kcache), _ptr(vcache), _ptr(q_start), B, n_q, Hq,
        Hkv, T_cap, float(sm_scale), _ptr(out), _dtype_code(out), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(stats), _stream(stream)))


def dq_prefill_attention_paged(tab: Tables, q: torch.Tensor, kpool: torch.Tensor, vpool: torch.Tensor,
                               page_table: torch.Tensor, q_start: torch.Tensor, out: torch.Tensor,
                               workspace: torch.Tensor | None = None, sm_scale: float | None = None,
                               stats: torch.Tensor | None = None, stream=None) -> None:
    """Chunked-prefill attention over page pools (see dq_prefill_attention)."""
    B, n_q, Hq, d = q.shape
    Hkv = kpool.shape[1]
    assert d == 128 and q.is_contiguous() and out.is_contiguous() and q_start.dtype == torch.int32
    assert page_table.dtype == torch.int32 and page_table.is_contiguous() and out.shape == q.shape
    if sm_scale is None:
        sm_scale = 128 ** -0.5
    workspace = _prefill_ws(tab, workspace, B, Hkv, 32 * page_table.shape[1], q.device, stream)
    _check("dq_prefill_attention_paged", load().dq_prefill_attention_paged(
        tab.handle, _ptr(q), _dtype_code(q), _ptr(kpool), _ptr(vpool), kpool.shape[0],
        _ptr(page_table), page_table.shape[1], _ptr(q_start), B, n_q, Hq, Hkv, float(sm_scale),
        _ptr(out), _dtype_code(out), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _ptr(stats), _stream(stream)))


def _check_cuda(names: str, *tensors) -> None:
    """Each tensor contiguous and on the current CUDA device (the calls take
    plain pointers). `names`: what the messages call them, in order."""
    device = tensors[0].get_device()
    for t in tensors:
        if t.get_device() != device or device < 0 or not t.is_contiguous():
            break
    else:
        if device == torch.cuda.current_device():
            return
        raise ValueError("the tensors are on cuda:%d, the current device is cuda:%d" % (device, torch.cuda.current_device()))
    for name, t in zip(names.split(), tensors):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("%s must be a contiguous CUDA tensor" % name)
        if t.get_device() != device:
            raise ValueError("%s is on %s, the others on cuda:%d" % (name, t.device, device))


def _check_int32(names: str, *pairs) -> None:
    """Each (tensor, shape): an int32 tensor of that shape."""
    for k, (t, shape) in enumerate(pairs):
        if t.dtype is not torch.int32 or t.shape != shape:
            raise ValueError("%s must be int32 %s, got %s %s" % (names.split()[k], shape, t.dtype, tuple(t.shape)))


def _check_stats(stats) -> None:
    """None, or room for a dq_stats on the current device (the kernels add to its fields)."""
    if stats is None:
        return
    if stats.nbytes < 8 * len(STATS_FIELDS) or stats.data_ptr() % 8:
        raise ValueError("stats must hold %d 64-bit counters (new_stats), got %s %s" % (len(STATS_FIELDS), stats.dtype, tuple(stats.shape)))
    _check_cuda("stats", stats)


def _check_heads(q, out, kcache, vcache) -> None:
    if q.shape[-1] != 128 or out.shape != q.shape:
        raise ValueError("q and out must have one shape with 128 coordinates, got %s and %s" % (tuple(q.shape), tuple(out.shape)))
    if kcache.dtype is not torch.uint8 or vcache.dtype is not torch.uint8:
        raise ValueError("caches must be uint8, got %s and %s" % (kcache.dtype, vcache.dtype))


def _check_shapes(what: str, k, v, k_shape, v_shape) -> None:
    if k.shape != k_shape or v.shape != v_shape:
        raise ValueError("%s must be %s and %s, got %s and %s" % (what, k_shape, v_shape, tuple(k.shape), tuple(v.shape)))


def _check_contiguous_cache(tab, B, kcache, vcache) -> None:
    T_cap = kcache.shape[-2]
    _check_shapes("caches", kcache, vcache, (B, tab.n_kv_heads, T_cap, tab.k.container_bytes),
                  (B, tab.n_kv_heads, T_cap, tab.v.container_bytes))


def _check_pools(tab, B, kpool, vpool, page_table) -> None:
    P = kpool.shape[0]
    _check_shapes("pools", kpool, vpool, (P, tab.n_kv_heads, tab.k.container_bytes, 32),
                  (P, tab.n_kv_heads, tab.v.container_bytes, 32))
    _check_int32("page_table", (page_table, (B, page_table.shape[-1])))


def dq_decode_attention_window(tab: Tables, q: torch.Tensor, kcache: torch.Tensor, vcache: torch.Tensor,
                               seq_lens: torch.Tensor, T_max: int, window: int, sinks: int, out: torch.Tensor,
                               workspace: torch.Tensor, sm_scale: float | None = None,
                               stats: torch.Tensor | None = None, stream=None) -> None:
    """dq_decode_attention over the last `window` tokens and the first `sinks`
    ones of each sequence; what lies between is never read."""
    _check_cuda("q kcache vcache seq_lens out workspace", q, kcache, vcache, seq_lens, out, workspace)
    _check_stats(stats)
    _check_heads(q, out, kcache, vcache)
    B, Hq, _ = q.shape
    _check_contiguous_cache(tab, B, kcache, vcache)
    _check_int32("seq_lens", (seq_lens, (B,)))
    if q.numel() == 0:
        return
    _check("dq_decode_attention_window", load().dq_decode_attention_window(
        tab.handle, q.data_ptr(), _dtype_code(q), kcache.data_ptr(), vcache.data_ptr(), seq_lens.data_ptr(), B, Hq, kcache.shape[1],
        kcache.shape[2], T_max, window, sinks, float(128 ** -0.5 if sm_scale is None else sm_scale), out.data_ptr(),
        _dtype_code(out), workspace.data_ptr(), workspace.nbytes, _addr(stats),
        _stream(stream)))


def dq_decode_attention_window_paged(tab: Tables, q: torch.Tensor, kpool: torch.Tensor, vpool: torch.Tensor,
                                     page_table: torch.Tensor, seq_lens: torch.Tensor, T_max: int, window: int,
                                     sinks: int, out: torch.Tensor, workspace: torch.Tensor,
                                     sm_scale: float | None = None, stats: torch.Tensor | None = None,
                                     stream=None) -> None:
    """dq_decode_attention_window over page pools; page-table entries between
    the first tokens and the window may be -1."""
    _check_cuda("q kpool vpool page_table seq_lens out workspace", q, kpool, vpool, page_table, seq_lens, out, workspace)
    _check_stats(stats)
    _check_heads(q, out, kpool, vpool)
    B, Hq, _ = q.shape
    _check_pools(tab, B, kpool, vpool, page_table)
    _check_int32("seq_lens", (seq_lens, (B,)))
    if q.numel() == 0:
        return
    _check("dq_decode_attention_window_paged", load().dq_decode_attention_window_paged(
        tab.handle, q.data_ptr(), _dtype_code(q), kpool.data_ptr(), vpool.data_ptr(), kpool.shape[0], page_table.data_ptr(),
        page_table.shape[1], seq_lens.data_ptr(), B, Hq, kpool.shape[1], T_max, window, sinks,
        float(128 ** -0.5 if sm_scale is None else sm_scale), out.data_ptr(), _dtype_code(out), workspace.data_ptr(),
        workspace.nbytes, _addr(stats), _stream(stream)))


def dq_prefill_window_workspace_bytes(tab: Tables, B: int, Hkv: int, T_cap: int, n_q: int, window: int,
                                      sinks: int) -> int:
    """Bytes of the dq_prefill_attention_window workspace (decoded tiles of what a chunk of n_q tokens sees)."""
    return int(load().dq_prefill_window_workspace_bytes(tab.handle, B, Hkv, T_cap, n_q, window, sinks))


def dq_prefill_attention_window(tab: Tables, q: torch.Tensor, kcache: torch.Tensor, vcache: torch.Tensor,
                                q_start: torch.Tensor, window: int, sinks: int, out: torch.Tensor,
                                workspace: torch.Tensor | None = None, sm_scale: float | None = None,
                                stats: torch.Tensor | None = None, stream=None) -> None:
    """dq_prefill_attention whose query at position p sees the tokens p -
    window + 1 .. p and the first `sinks` ones; workspace uint8 of
    dq_prefill_window_workspace_bytes (allocated if None)."""
    _check_cuda("q kcache vcache q_start out", q, kcache, vcache, q_start, out)
    _check_stats(stats)
    _check_heads(q, out, kcache, vcache)
    B, n_q, Hq, _ = q.shape
    _check_contiguous_cache(tab, B, kcache, vcache)
    _check_int32("q_start", (q_start, (B,)))
    if q.numel() == 0:
        return
    if workspace is None:
        workspace = _workspace_for(dq_prefill_window_workspace_bytes(tab, B, kcache.shape[1], kcache.shape[2], n_q,
                                                                     window, sinks), q.device, stream)
    else:
        _check_cuda("q workspace", q, workspace)
        if stream is not None:  # (the caller may drop it before the kernels run)
            workspace.record_stream(stream)
    _check("dq_prefill_attention_window", load().dq_prefill_attention_window(
        tab.handle, q.data_ptr(), _dtype_code(q), kcache.data_ptr(), vcache.data_ptr(), q_start.data_ptr(), B, n_q, Hq, kcache.shape[1],
        kcache.shape[2], window, sinks, float(128 ** -0.5 if sm_scale is None else sm_scale), out.data_ptr(),
        _dtype_code(out), workspace.data_ptr(), workspace.nbytes, _addr(stats),
        _stream(stream)))


def dq_prefill_attention_window_paged(tab: Tables, q: torch.Tensor, kpool: torch.Tensor, vpool: torch.Tensor,
                                      page_table: torch.Tensor, q_start: torch.Tensor, window: int, sinks: int,
                                      out: torch.Tensor, workspace: torch.Tensor | None = None,
                                      sm_scale: float | None = None, stats: torch.Tensor | None = None,
                                      stream=None) -> None:
    """dq_prefill_attention_window over page pools; page-table entries that no
    query of the chunk sees may be -1."""
    _check_cuda("q kpool vpool page_table q_start out", q, kpool, vpool, page_table, q_start, out)
    _check_stats(stats)
    _check_heads(q, out, kpool, vpool)
    B, n_q, Hq, _ = q.shape
    _check_pools(tab, B, kpool, vpool, page_table)
    _check_int32("q_start", (q_start, (B,)))
    if q.numel() == 0:
        return
    if workspace is None:
        workspace = _workspace_for(dq_prefill_window_workspace_bytes(tab, B, kpool.shape[1], 32 * page_table.shape[1],
                                                                     n_q, window, sinks), q.device, stream)
    else:
        _check_cuda("q workspace", q, workspace)
        if stream is not None:  # (the caller may drop it before the kernels run)
            workspace.record_stream(stream)
    _check("dq_prefill_attention_window_paged", load().dq_prefill_attention_window_paged(
        tab.handle, q.data_ptr(), _dtype_code(q), kpool.data_ptr(), vpool.data_ptr(), kpool.shape[0], page_table.data_ptr(),
        page_table.shape[1], q_start.data_ptr(), B, n_q, Hq, kpool.shape[1], window, sinks,
        float(128 ** -0.5 if sm_scale is None else sm_scale), out.data_ptr(), _dtype_code(out), workspace.data_ptr(),
        workspace.nbytes, _addr(stats), _stream(stream)))


def new_page_state(num_pages: int, B: int, max_pages: int, device=None):
    """(refs [num_pages], page_table [B, max_pages], lens [B]) of an empty paged cache, int32."""
    device = device or "cuda"
    return (torch.zeros(num_pages, dtype=torch.int32, device=device),
            torch.full((B, max_pages), -1, dtype=torch.int32, device=device),
            torch.zeros(B, dtype=torch.int32, device=device))


def new_page_counts(device=None) -> torch.Tensor:
    """A zeroed device dq_page_counts (one int32 per field of PAGE_COUNT_FIELDS)."""
    return torch.zeros(len(PAGE_COUNT_FIELDS), dtype=torch.int32, device=device or "cuda")


def page_counts_dict(counts: torch.Tensor) -> dict:
    return dict(zip(PAGE_COUNT_FIELDS, counts.cpu().tolist()))


def dq_pages_workspace_bytes(tab: Tables, num_pages: int, B: int, max_pages: int) -> int:
    """Bytes of the workspace of dq_pages_advance, _fork and _compact for tables of at most B rows."""
    return int(load().dq_pages_workspace_bytes(tab.handle, num_pages, B, max_pages))


def dq_pages_advance(tab: Tables, refs: torch.Tensor, page_table: torch.Tensor, lens: torch.Tensor,
                     n_new: torch.Tensor, refs_out: torch.Tensor, page_table_out: torch.Tensor,
                     lens_out: torch.Tensor, counts: torch.Tensor, workspace: torch.Tensor, window: int = 0,
                     sinks: int = 0, stream=None) -> None:
    """The pages of the next n_new[b] tokens of every sequence (n_new[b] < 0:
    the sequence ends); with a window the pages behind it go back. int32: refs
    [num_pages], page_table [B, max_pages], lens and n_new [B]; the outputs may
    be the inputs."""
    _check_cuda("refs page_table lens n_new refs_out page_table_out lens_out counts workspace", refs, page_table, lens,
                n_new, refs_out, page_table_out, lens_out, counts, workspace)
    B, max_pages = rows = page_table.shape
    P = refs.numel()
    _check_int32("refs page_table lens n_new refs_out page_table_out lens_out counts", (refs, (P,)), (page_table, rows),
                 (lens, (B,)), (n_new, (B,)), (refs_out, (P,)), (page_table_out, rows), (lens_out, (B,)), (counts, (8,)))
    _check("dq_pages_advance", load().dq_pages_advance(
        tab.handle, P, refs.data_ptr(), page_table.data_ptr(), max_pages, lens.data_ptr(), n_new.data_ptr(), B, window, sinks,
        refs_out.data_ptr(), page_table_out.data_ptr(), lens_out.data_ptr(), counts.data_ptr(), workspace.data_ptr(),
        workspace.nbytes, _stream(stream)))


def dq_pages_fork(tab: Tables, refs: torch.Tensor, page_table: torch.Tensor, lens: torch.Tensor,
                  parent: torch.Tensor, refs_out: torch.Tensor, page_table_out: torch.Tensor,
                  lens_out: torch.Tensor, pairs: torch.Tensor, counts: torch.Tensor, workspace: torch.Tensor,
                  stream=None) -> None:
    """Row c of the new table [B_out, max_pages] is row parent[c] of the old
    one (negative: empty). Pages are shared, but for those that the row will
    write to; pairs [B_out, 2] lists the copies of partly filled last pages for
    dq_pages_copy. Outputs must be other tensors than the inputs."""
    _check_cuda("refs page_table lens parent refs_out page_table_out lens_out pairs counts workspace", refs, page_table,
                lens, parent, refs_out, page_table_out, lens_out, pairs, counts, workspace)
    B, max_pages = rows = page_table.shape
    P, B_out = refs.numel(), parent.numel()
    _check_int32("refs page_table lens parent refs_out page_table_out lens_out pairs counts", (refs, (P,)),
                 (page_table, rows), (lens, (B,)), (parent, (B_out,)), (refs_out, (P,)),
                 (page_table_out, (B_out, max_pages)), (lens_out, (B_out,)), (pairs, (B_out, 2)), (counts, (8,)))
    _check("dq_pages_fork", load().dq_pages_fork(
        tab.handle, P, refs.data_ptr(), page_table.data_ptr(), max_pages, lens.data_ptr(), B, parent.data_ptr(), B_out, refs_out.data_ptr(),
        page_table_out.data_ptr(), lens_out.data_ptr(), pairs.data_ptr(), counts.data_ptr(), workspace.data_ptr(),
        workspace.nbytes, _stream(stream)))


def dq_pages_compact(tab: Tables, refs: torch.Tensor, page_table: torch.Tensor, refs_out: torch.Tensor,
                     page_table_out: torch.Tensor, pairs: torch.Tensor, counts: torch.Tensor,
                     workspace: torch.Tensor, stream=None) -> None:
    """Renumbers the pages in use to the lowest numbers; pairs [max(1,
    num_pages // 2), 2] lists the moves for dq_pages_copy. The outputs may be
    the inputs."""
    _check_cuda("refs page_table refs_out page_table_out pairs counts workspace", refs, page_table, refs_out,
                page_table_out, pairs, counts, workspace)
    B, max_pages = rows = page_table.shape
    P = refs.numel()
    _check_int32("refs page_table refs_out page_table_out pairs counts", (refs, (P,)), (page_table, rows),
                 (refs_out, (P,)), (page_table_out, rows), (pairs, (max(1, P // 2), 2)), (counts, (8,)))
    _check("dq_pages_compact", load().dq_pages_compact(
        tab.handle, P, refs.data_ptr(), page_table.data_ptr(), max_pages, B, refs_out.data_ptr(), page_table_out.data_ptr(), pairs.data_ptr(),
        counts.data_ptr(), workspace.data_ptr(), workspace.nbytes, _stream(stream)))


def dq_pages_copy(tab: Tables, kpool: torch.Tensor, vpool: torch.Tensor, pairs: torch.Tensor,
                  counts: torch.Tensor | None = None, stats: torch.Tensor | None = None, stream=None) -> None:
    """Copies the pages that pairs int32 [n, 2] names (source, destination) in
    pools [num_pages, Hkv, C, 32], or [layers, num_pages, Hkv, C, 32] (each
    layer contiguous): the first counts.pairs of them, or all."""
    layers, P = (kpool.shape[0], kpool.shape[1]) if kpool.dim() == 5 else (1, kpool.shape[0])
    lead = (layers, P) if kpool.dim() == 5 else (P,)
    _check_shapes("pools", kpool, vpool, (*lead, tab.n_kv_heads, tab.k.container_bytes, 32),
                  (*lead, tab.n_kv_heads, tab.v.container_bytes, 32))
    if kpool.dtype is not torch.uint8 or vpool.dtype is not torch.uint8:
        raise ValueError("pools must be uint8, got %s and %s" % (kpool.dtype, vpool.dtype))
    if layers == 0:
        return
    k0, v0 = (x if x.is_contiguous() or x.dim() == 4 else x[0] for x in (kpool, vpool))
    _check_cuda("kpool vpool pairs", k0, v0, pairs)
    _check_int32("pairs", (pairs, (pairs.shape[0], 2)))
    if counts is not None:
        _check_cuda("counts pairs", counts, pairs)
        _check_int32("counts", (counts, (8,)))
    _check_stats(stats)
    _check("dq_pages_copy", load().dq_pages_copy(
        tab.handle, kpool.data_ptr(), vpool.data_ptr(), P, layers, kpool.stride(0), vpool.stride(0), pairs.data_ptr(),
        pairs.shape[0], _addr(counts), _addr(stats), _stream(stream)))


def dq_decode_symbols(tab: Tables, cache: torch.Tensor, kind: int, syms: torch.Tensor,
                      norm16: torch.Tensor, status: torch.Tensor | None = None,
                      stats: torch.Tensor | None = None, stream=None) -> None:
    """cache uint8 [..., C] (flat containers); syms uint8 [n, 128]; norm16 int16/uint16 [n]."""
    n = syms.shape[0]
    _check("dq_decode_symbols", load().dq_decode_symbols(
        tab.handle, _ptr(cache), kind, n, _ptr(syms), _ptr(norm16), _ptr(status), _ptr(stats),
        _stream(stream)))


def dq_error_string(code: int) -> str:
    return load().dq_error_string(code).decode()


def dq_design_stream(n_levels: int, container_bytes: int, rate_offset: float = 0.0) -> dict:
    """Host-only table design of one stream (no device needed)."""
    lev = (C.c_float * 8)(); thr = (C.c_float * 7)(); f = (C.c_uint32 * 8)()
    cum = (C.c_uint32 * 9)(); cost = (C.c_float * 8)()
    lam = C.c_double(); ent = C.c_double(); mse = C.c_double()
    _check("dq_design_stream", load().dq_design_stream(
        n_levels, container_bytes, rate_offset, lev, thr, f, cum, cost, C.byref(lam),
        C.byref(ent), C.byref(mse)))
    n = n_levels
    return dict(levels=list(lev)[:n], thresholds=list(thr)[:n - 1], freq=list(f)[:n],
                cum=list(cum)[:n + 1], cost=list(cost)[:n], lam=lam.value, entropy=ent.value,
                mse=mse.value)


def new_pool(num_pages: int, Hkv: int, C: int, device=None) -> torch.Tensor:
    """Zeroed uint8 page pool [num_pages, Hkv, C, 32] (pages of 32 tokens)."""
    return torch.zeros((num_pages, Hkv, C, 32), dtype=torch.uint8, device=device or "cuda")


def dq_append_kv_paged(tab: Tables, k: torch.Tensor, v: torch.Tensor, start_pos: torch.Tensor,
                       kpool: torch.Tensor, vpool: torch.Tensor, page_table: torch.Tensor,
                       stats: torch.Tensor | None = None, stream=None,
                       workspace: torch.Tensor | None = None) -> None:
    """Append into page pools [num_pages, Hkv, C, 32] through page_table
    int32 [B, max_pages] (see dq_append_kv for the other arguments)."""
    B, Hkv, n_new, d = k.shape
    assert d == 128 and v.shape == k.shape and k.dtype == v.dtype
    assert k.is_contiguous() and v.is_contiguous() and kpool.is_contiguous() and vpool.is_contiguous()
    assert page_table.dtype == torch.int32 and page_table.is_contiguous() and page_table.shape[0] == B
    if workspace is None:
        nbytes = dq_append_workspace_bytes(tab, B, Hkv, n_new)
        workspace = _workspace_for(max(nbytes, 16), kpool.device, stream)
    _check("dq_append_kv_paged", load().dq_append_kv_paged(
        tab.handle, _ptr(k), _ptr(v), _dtype_code(k), B, Hkv, n_new, _ptr(start_pos),
        _ptr(kpool), _ptr(vpool), kpool.shape[0], _ptr(page_table), page_table.shape[1],
        _ptr(workspace), workspace.numel(), _ptr(stats), _stream(stream)))


def dq_decode_attention_paged(tab: Tables, q: torch.Tensor, kpool: torch.Tensor, vpool: torch.Tensor,
                              page_table: torch.Tensor, seq_lens: torch.Tensor, T_max: int,
                              out: torch.Tensor, workspace: torch.Tensor, sm_scale: float | None = None,
                              stats: torch.Tensor | None = None, stream=None) -> None:
    """Decode attention over page pools (see dq_decode_attention)."""
    B, Hq, d = q.shape
    Hkv = kpool.shape[1]
    assert d == 128 and q.is_contiguous() and out.is_contiguous() and seq_lens.dtype == torch.int32
    assert page_table.dtype == torch.int32 and page_table.is_contiguous()
    if sm_scale is None:
        sm_scale = 128 ** -0.5
    _check("dq_decode_attention_paged", load().dq_decode_attention_paged(
        tab.handle, _ptr(q), _dtype_code(q), _ptr(kpool), _ptr(vpool), kpool.shape[0],
        _ptr(page_table), page_table.shape[1], _ptr(seq_lens), B, Hq, Hkv, T_max, float(sm_scale),
        _ptr(out), _dtype_code(out), _ptr(workspace), workspace.numel(), _ptr(stats),
        _stream(stream)))
