"""Calls of the drafted rows' attention one behind the other, each on the last one's output: the next
grid starts early, and reads nothing before the last one has ended."""

import pytest
import torch

import test_tree_gpu
from gqa_attention_kv_decode_gb300 import binding

pytestmark = pytest.mark.gpu
CALLS = 24


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("B,Hq,Hkv,D,Tq,L", [(1, 14, 2, 64, 8, 100), (8, 32, 8, 128, 8, 128), (3, 8, 1, 128, 40, 120),
                                             (200, 8, 2, 64, 5, 90), (1, 14, 2, 64, 8, 513), (2, 8, 1, 128, 40, 3000),
                                             (30, 8, 2, 64, 9, 2000)])
@pytest.mark.parametrize("captured", [False, True])
def test_each_reads_the_last_ones_output(B, Hq, Hkv, D, Tq, L, captured):
    """One tile a unit (one grid a call), clusters, and the list with its merge; two workspaces in turn."""
    c = test_tree_gpu.Case(B, Hq, Hkv, D, Tq, test_tree_gpu.lens_of(B, Tq, L, 1), seed=4)
    args, ws, out = c.args(), [c.workspace() for _ in range(2)], [torch.zeros_like(c.q) for _ in range(CALLS)]

    def calls(wait):
        q = c.q
        for i, o in enumerate(out):
            binding.gqa_attn_decode_tree(q, c.k, c.v, *args, o, 4 * c.scale, ws[i % 2], L)
            q = o
            if wait:
                torch.cuda.synchronize()

    calls(True)
    want = [o.clone() for o in out]
    graph = None
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            calls(False)
    for _ in range(5):
        for o in out:
            o.zero_()
        if captured:
            graph.replay()
        else:
            calls(False)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    assert all(torch.isfinite(o).all() for o in want)
