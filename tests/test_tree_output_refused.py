"""A refused convenience call on a stream of its own gives its output back while the fill of it may
still run there: the current stream, which gets the memory, waits for it (CPU, with stand-ins)."""

import contextlib

import pytest
import torch

from gqa_attention_kv_decode_gb300 import binding


class Stream:
    def __init__(self, name, log):
        self.name, self.log = name, log

    def wait_stream(self, other):
        self.log.append((self.name, "waits for", other.name))


@pytest.mark.parametrize("name", ["decode_tree", "decode_tree_paged"])
@pytest.mark.parametrize("stream", [None, 77777, 1])
def test_the_current_stream_waits_for_the_fill(monkeypatch, name, stream):
    import __graft_entry__
    __graft_entry__.build()
    log = []
    on = [Stream("current", log)]

    @contextlib.contextmanager
    def use(s):
        on.append(s)
        try:
            yield
        finally:
            on.pop()

    def refuse(*a, **kw):
        raise ValueError("refused")

    monkeypatch.setattr(torch.cuda, "stream", use)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: on[-1])
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle: Stream(handle, log))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda: Stream("default", log))
    # (nothing may need the stream after the call: a caller's own one may be gone by then)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda *a: log.append("record_stream"))
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: True))
    monkeypatch.setattr(binding, "gqa_attn_" + name, refuse)
    q, ws = torch.ones((2, 8, 4, 64), dtype=torch.bfloat16), torch.zeros(1 << 20, dtype=torch.uint8)
    k, table, lens = (torch.zeros((2, 2, 64, 64), dtype=torch.bfloat16), torch.zeros((2, 1), dtype=torch.int32),
                      torch.full((2,), 9, dtype=torch.int32))
    with pytest.raises(ValueError, match="refused"):
        getattr(binding, name)(*((q, k, k, lens) if name == "decode_tree" else (q, k, k, table, lens)), workspace=ws,
                               stream=stream)
    assert log == ([] if stream is None else [("current", "waits for", "default" if stream == 1 else stream)])
    monkeypatch.setattr(binding, "gqa_attn_" + name, lambda *a, **kw: None)
    log.clear()
    getattr(binding, name)(*((q, k, k, lens) if name == "decode_tree" else (q, k, k, table, lens)), workspace=ws,
                           stream=stream)
    assert log == []
