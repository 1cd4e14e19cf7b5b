"""A workspace that a call allocates for itself comes from the pool of the
stream that the call runs on."""
import contextlib
import types

import pytest
import torch

import decode_attention_dq_b200 as dq
from decode_attention_dq_b200 import _native as N
from decode_attention_dq_b200 import synth
from tests import _common as cm


def _calls(tab, k, q, start, kc, kp, vc, vp, table, out, stream):
    """Every call that allocates a workspace when it is given none."""
    return {
        "append": lambda: dq.dq_append_kv(tab, k, k, start, kc, vc, stream=stream),
        "append_paged": lambda: dq.dq_append_kv_paged(tab, k, k, start, kp, vp, table, stream=stream),
        "prefill": lambda: dq.dq_prefill_attention(tab, q, kc, vc, start, out, stream=stream),
        "prefill_paged": lambda: dq.dq_prefill_attention_paged(tab, q, kp, vp, table, start, out, stream=stream),
        "prefill_window": lambda: dq.dq_prefill_attention_window(tab, q, kc, vc, start, 40, 4, out, stream=stream),
        "prefill_window_paged": lambda: dq.dq_prefill_attention_window_paged(tab, q, kp, vp, table, start, 40, 4, out,
                                                                             stream=stream),
    }


NAMES = ("append", "append_paged", "prefill", "prefill_paged", "prefill_window", "prefill_window_paged")


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("given", [False, True])
def test_allocation_happens_on_the_calls_stream(monkeypatch, name, given):
    # No GPU: a library that accepts everything, and a record of the stream that is current at each allocation.
    current, seen = [None], []
    real_empty = torch.empty

    @contextlib.contextmanager
    def on(stream):
        current.append(stream)
        yield
        current.pop()

    def empty(*a, **kw):
        seen.append(current[-1])
        return real_empty(*a, **kw)

    class Lib:
        def __getattr__(self, call):
            return lambda *a: 64 if call.endswith("_bytes") else 0

    stream = types.SimpleNamespace(cuda_stream=5) if given else None
    stream_table = types.SimpleNamespace(container_bytes=36)
    tab = types.SimpleNamespace(handle=None, n_kv_heads=2, k=stream_table, v=stream_table)
    k, q = torch.zeros(1, 2, 8, 128), torch.zeros(1, 8, 4, 128)
    kc, kp = torch.zeros(1, 2, 64, 36, dtype=torch.uint8), torch.zeros(2, 2, 36, 32, dtype=torch.uint8)
    start, table = torch.zeros(1, dtype=torch.int32), torch.zeros(1, 2, dtype=torch.int32)
    call = _calls(tab, k, q, start, kc, kp, kc.clone(), kp.clone(), table, torch.zeros_like(q), stream)[name]
    monkeypatch.setattr(N, "load", lambda: Lib())
    monkeypatch.setattr(N, "_check_cuda", lambda *a: None)
    monkeypatch.setattr(N, "_stream", lambda s: None)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch, "empty", empty)
    call()
    assert seen == [stream]


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_a_block_just_freed_on_the_current_stream_stays_whole(name):
    # The current stream still has to read a block that Python has let go of, and the call runs on another stream.
    B, Hkv, G, T, n = 2, 2, 4, 512, 256
    w = synth.scaled(synth.WORKLOADS["qwen3_8b_b16_t8k"], B=B, Hkv=Hkv, Hq=Hkv * G, T=T)
    K, _, _ = cm.inputs(w)
    tab = cm.lib_tables(Hkv, v_levels=8)
    kc, _ = cm.gpu_append_all(tab, K, K, torch.bfloat16)
    k = torch.from_numpy(K[:, :, :n]).cuda().contiguous()
    q = torch.from_numpy(synth.q_chunk(w, n)).cuda()
    start = torch.full((B,), T - n, dtype=torch.int32, device="cuda")
    table = torch.arange(B * T // 32, dtype=torch.int32, device="cuda").reshape(B, -1)
    kp = kc.reshape(B, Hkv, T // 32, 36, 32).transpose(1, 2).reshape(-1, Hkv, 36, 32).contiguous()
    vc, vp = kc.clone(), kp.clone()
    want = torch.empty_like(q)
    _calls(tab, k, q, start, kc, kp, vc, vp, table, want, None)[name]()
    torch.cuda.synchronize()
    side, out = torch.cuda.Stream(), torch.empty_like(q)
    sizes = [N.dq_append_workspace_bytes(tab, B, Hkv, n), N.dq_prefill_workspace_bytes(tab, B, Hkv, T),
             N.dq_prefill_window_workspace_bytes(tab, B, Hkv, T, n, 40, 4)]
    blocks = [torch.full((s,), 7, dtype=torch.uint8, device="cuda") for s in sizes for _ in range(3)]
    torch.cuda.synchronize()
    torch.cuda._sleep(40_000_000)
    later = [x.clone() for x in blocks]
    del blocks
    _calls(tab, k, q, start, kc, kp, vc, vp, table, out, side)[name]()
    side.synchronize()
    torch.cuda.synchronize()
    assert all(bool((x == 7).all()) for x in later)
    if name.startswith("prefill"):
        assert torch.equal(out, want)
