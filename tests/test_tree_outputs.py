"""The outputs that the convenience calls of the drafted rows' attention make themselves: rows that no
query belongs to are zeros, on the call's stream (CPU, with stand-ins; GPU, over memory that held NaN)."""

import contextlib

import numpy as np
import pytest
import torch

import oracle
import parity
from gqa_attention_kv_decode_gb300 import binding, inputs

B, HQ, HKV, TQ, D, S = 3, 8, 2, 4, 64, 128



@pytest.mark.parametrize("name", ["decode_tree", "decode_tree_paged"])
@pytest.mark.parametrize("stream", [None, 77777, 0])
def test_rows_that_are_not_written_are_zeros(monkeypatch, name, stream):
    import __graft_entry__
    __graft_entry__.build()
    on, filled = ["current"], []

    @contextlib.contextmanager
    def use(s):
        on.append(s)
        yield
        on.pop()

    monkeypatch.setattr(torch.cuda, "stream", use)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle: handle)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda: "default")
    zero_ = torch.Tensor.zero_
    monkeypatch.setattr(torch.Tensor, "zero_", lambda t: (filled.append(on[-1]), zero_(t))[1])
    empty_like = torch.empty_like
    made = []

    def dirty(t, **kw):
        made.append(on[-1])
        return empty_like(t, **kw).fill_(float("nan"))

    monkeypatch.setattr(torch, "empty_like", dirty)
    monkeypatch.setattr(binding, "gqa_attn_" + name, lambda *a, **kw: None)
    q, ws = torch.ones((B, HQ, TQ, D), dtype=torch.bfloat16), torch.zeros(1 << 20, dtype=torch.uint8)
    k = torch.zeros((B, HKV, S, D) if name == "decode_tree" else (6, HKV, 64, D), dtype=torch.bfloat16)
    lens, table = torch.full((B,), 9, dtype=torch.int32), torch.zeros((B, 2), dtype=torch.int32)
    args = (q, k, k, lens) if name == "decode_tree" else (q, k, k, table, lens)
    o = getattr(binding, name)(*args, workspace=ws, stream=stream)
    assert o.shape == q.shape and o.dtype == q.dtype and not o.any()
    # memory of the current stream, as every output; filled where the call's kernels follow
    assert made == ["current"]
    assert filled == ["current" if stream is None else "default" if stream == 0 else stream]


@pytest.mark.gpu
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("side", [False, True])
def test_rows_past_the_queries(paged, side):
    """Fewer queries than Tq, none at all, and requests shorter than Tq without q_lens."""
    import __graft_entry__
    __graft_entry__.build()
    dev, dt = "cuda", torch.bfloat16
    q = inputs.randn((B, HQ, TQ, D), 1, dt, dev)
    k, v = (inputs.randn((B, HKV, S, D), s, dt, dev) for s in (2, 3))
    kp, vp = (x.view(B, HKV, 2, 64, D).transpose(1, 2).reshape(2 * B, HKV, 64, D).contiguous() for x in (k, v))
    table = torch.arange(2 * B, dtype=torch.int32, device=dev).view(B, 2)
    stream = torch.cuda.Stream() if side else None
    for lens, q_lens in (([100, 3, 0], None), ([100, 90, 128], [1, 0, 4]), ([100, 2, 0], [4, 2, 0])):
        kl, ql = (None if x is None else torch.tensor(x, dtype=torch.int32, device=dev) for x in (lens, q_lens))
        poison = torch.full_like(q, float("nan"))
        torch.cuda.synchronize()
        del poison  # (the next output of this size is its memory)
        if paged:
            o = binding.decode_tree_paged(q, kp, vp, table, kl, q_lens=ql, stream=stream)
        else:
            o = binding.decode_tree(q, k, v, kl, q_lens=ql, stream=stream)
        torch.cuda.synchronize()
        f = lambda t: t.float().cpu().numpy()  # noqa: E731
        ref, _ = oracle.attention_tree(f(q), f(k), f(v), None, q_lens, None, lens, D ** -0.5, np.zeros(q.shape))
        parity.check(f(o), ref, "bf16")
        for b in range(B):
            n = min(TQ if q_lens is None else q_lens[b], lens[b])
            assert not o[b, :, n:].any()
