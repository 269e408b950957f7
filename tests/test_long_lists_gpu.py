"""Lists longer than one pass takes: page copies of more than 1,024 entries, and paged attention of
drafted rows of more than 1,024 requests (launches of their own, each with its part of the table)."""

import numpy as np
import pytest
import torch

from gqa_attention_kv_decode_gb300 import binding, inputs
from test_pages_gpu import run_copy, ws  # noqa: F401  (ws: a fixture)
from test_tree_gpu import Case, lens_of

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


# (heads of up to 4 KB in a block by sixteen warps, up to 8 KB by eight, above by four)
@pytest.mark.parametrize("bs,D,Hkv,layers", [(16, 64, 2, 1), (64, 64, 1, 2), (80, 128, 1, 1)])
@pytest.mark.parametrize("n", [1023, 1024, 1025, 2500])
@pytest.mark.parametrize("live", [1.0, 0.02])
def test_copies_of_long_lists(ws, bs, D, Hkv, layers, n, live):  # noqa: F811
    r = np.random.default_rng(n)
    pool = n + 300
    order = r.permutation(pool)
    src = order[r.integers(0, 300, n)]  # (blocks that are copied more than once, and none that is written)
    dst, rows = order[300:], r.integers(1, bs + 1, n)
    on = r.random(n) < live
    for i in (0, 1022, 1023, 1024, 1025, 2047, 2048, n - 1):  # at the borders of the passes
        if i < n:
            on[i] = True
    src = np.where(on, src, -1)
    k, v = (inputs.randn((layers, pool, Hkv, bs, D), s, torch.bfloat16, DEV) for s in (1, 2))
    assert run_copy(ws, src, dst, rows, k, v) == 0
    assert run_copy(ws, src, dst, None, k, v) == 0


def test_a_bad_entry_of_a_later_pass(ws):  # noqa: F811
    n = 2100
    src, dst = np.full(n, -1), np.full(n, -1)
    src[[3, 1500, 2099]], dst[[3, 1500, 2099]] = [0, 1, 2], [4, 99, 5]
    k, v = (inputs.randn((1, 6, 2, 16, 64), s, torch.bfloat16, DEV) for s in (1, 2))
    assert run_copy(ws, src, dst, None, k, v) == binding.GQA_DEV_BAD_BLOCK


@pytest.mark.parametrize("B", [1024, 1025, 2500])
@pytest.mark.parametrize("mask", ["tree", None])
def test_paged_requests_of_several_launches(B, mask):
    lens = lens_of(B, 0, 150, 5)
    ql = np.minimum(np.random.default_rng(8).integers(0, 4, B), lens)
    Case(B, 4, 2, 64, 3, lens, ql, mask=mask, seed=5).check(64)
