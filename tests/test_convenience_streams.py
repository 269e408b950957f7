"""The workspace that a convenience call makes for itself belongs to the stream
that the call runs on (CPU, with stand-ins for the library's calls), and calls
on a stream of their own are right while the current stream makes and fills
tensors (GPU)."""

import contextlib

import pytest
import torch

from gqa_attention_kv_decode_gb300 import binding, inputs

B, HQ, HKV, D, S = 2, 8, 2, 64, 70


def tensors(device="cpu", dtype=torch.bfloat16):
    def r(*shape):
        return torch.zeros(shape, dtype=dtype, device=device)
    q, k = r(B, HQ, 1, D), r(B, HKV, S, D)
    pool, table = r(6, HKV, 64, D), torch.zeros((B, 2), dtype=torch.int32, device=device)
    codes, sb = torch.zeros((B, HKV, S, D // 2), dtype=torch.uint8), torch.zeros((B, HKV, S, 1), dtype=torch.float16)
    lens = torch.full((B,), S, dtype=torch.int32, device=device)
    return {
        "decode": (q, k, k),
        "decode_paged": (q, pool, pool, table, lens, 128),
        "decode_shared_prefix": (q, k[0], k[0], k, k),
        "decode_shared_prefix_paged": (q, pool, pool, table[0], table, lens, 128, 128),
        "decode_q4": (q, codes, sb, sb, codes, sb, sb),
        "decode_q4_residual": (q, codes, sb, sb, codes, sb, sb, k, k, lens, lens),
    }


@pytest.mark.parametrize("name", list(tensors()))
@pytest.mark.parametrize("stream", [None, 77777, 0, 1, 2])
def test_the_workspace_is_made_on_the_calls_stream(monkeypatch, name, stream):
    import __graft_entry__
    __graft_entry__.build()
    on, seen = ["current"], []

    @contextlib.contextmanager
    def use(s):
        on.append(s)
        yield
        on.pop()

    monkeypatch.setattr(torch.cuda, "stream", use)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle: handle)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda: "default")
    zeros = torch.zeros
    monkeypatch.setattr(torch, "zeros", lambda *a, **kw: (seen.append(on[-1]), zeros(*a, **kw))[1])
    monkeypatch.setattr(binding, "gqa_attn_" + name, lambda *a, **kw: None)
    args = tensors()[name]
    seen.clear()
    o = getattr(binding, name)(*args, stream=stream)
    assert o.shape == args[0].shape
    assert seen == ["current" if stream is None else "default" if stream <= 2 else stream]
    seen.clear()
    getattr(binding, name)(*args, stream=stream, workspace=zeros(1 << 20, dtype=torch.uint8))
    assert seen == []


@pytest.mark.gpu
@pytest.mark.parametrize("as_handle", [False, True])
def test_calls_on_a_stream_while_the_current_one_fills_tensors(as_handle):
    import __graft_entry__
    __graft_entry__.build()
    dev, dt = "cuda", torch.bfloat16
    q = inputs.randn((40, 28, 1, 128), 5, dt, dev)
    k, v = (inputs.randn((40, 4, 600, 128), s, dt, dev) for s in (6, 7))
    kp, vp = (inputs.randn((4, 3000, 128), s, dt, dev) for s in (8, 9))
    s = torch.cuda.Stream()
    stream = s.cuda_stream if as_handle else s
    want = [binding.decode(q, k, v), binding.decode_shared_prefix(q, kp, vp, k, v)]
    n = max(binding.gqa_attn_decode_workspace_size(40, 28, 4, 128, 600, binding.GQA_BF16),
            binding.gqa_attn_decode_shared_prefix_workspace_size(40, 28, 4, 128, 3000, 600))
    torch.cuda.synchronize()
    for _ in range(20):
        got = []
        for call in (lambda: binding.decode(q, k, v, stream=stream),
                     lambda: binding.decode_shared_prefix(q, kp, vp, k, v, stream=stream)):
            s.wait_stream(torch.cuda.current_stream())  # (the output is the current stream's)
            got.append(call())
            for size in (n, n // 2, n // 3):  # (of the sizes that a freed workspace serves)
                torch.full((size,), 0xFF, dtype=torch.uint8, device=dev)
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
