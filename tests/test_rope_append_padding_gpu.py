"""gqa_attn_rope_append where most tokens are padding, on a stream of its own
and in a graph: every output against the oracle element by element, the rows
that no token names bit for bit, and the status (bounds: test_rope_append_gpu)."""

import pytest
import torch

from gqa_attention_kv_decode_gb300 import binding
from test_rope_append_gpu import Case, check

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,Hq,Hkv,D", [(40000, 2, 2, 64), (9000, 6, 2, 128)])
@pytest.mark.parametrize("which", ["both", "slots", "q_slots"])
def test_long_runs_of_padding(T, Hq, Hkv, D, dtype, which):
    """Whole blocks with nothing to do, with K and V alone and with Q alone."""
    c = Case(T, Hq, Hkv, D, dtype, bs=64, seed=22)
    if which != "q_slots":
        c.slots[100:T - 1000] = -1
    if which != "slots":
        c.q_slots[90:T - 500] = -1
    check(c)


@pytest.mark.parametrize("T,kind", [(1, {}), (64, dict(pad=5)), (500, dict(adjacent=True)), (3000, dict(rot=48, pad=40))])
@pytest.mark.parametrize("Hq,Hkv,D", [(32, 8, 128), (14, 2, 64)])
def test_every_output_on_another_stream(T, kind, Hq, Hkv, D):
    s = torch.cuda.Stream()
    c = Case(T, Hq, Hkv, D, torch.bfloat16, bs=64, seed=14, **kind)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        check(c, ws, stream=s)


def test_replayed_with_other_places():
    """A captured call follows the places, positions and values of its buffers."""
    c = Case(700, 28, 4, 128, torch.bfloat16, bs=64, seed=30)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    c.call(ws)  # (one-time kernel setup)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.call(ws)
    for seed in (31, 32):
        other = Case(700, 28, 4, 128, torch.bfloat16, bs=64, seed=seed, pad=seed)
        for name in ("q", "k", "v", "wq", "wk", "pos", "slots", "q_slots", "q_out", "kc", "vc"):
            getattr(c, name).copy_(getattr(other, name))
        c.call = lambda ws, **kw: g.replay()
        check(c, ws)
    assert binding.gqa_attn_read_device_status(ws) == 0
