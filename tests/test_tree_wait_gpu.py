"""The lost-copy path of the drafted rows' attention and of the page copies (see
test_wait_timeout_gpu.py): reported, and the next call on the same context is right."""

import numpy as np
import pytest
import torch

import parity
import test_tree_gpu
from gqa_attention_kv_decode_gb300 import binding, inputs

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Tq", [5, 50])
def test_tree_lost_copy_is_reported_and_the_context_survives(D, Tq):
    """Two slots of their own, and a pair of row tiles."""
    c = test_tree_gpu.Case(3, 16, 4, D, Tq, [3000, 700, 90])
    ws = c.workspace()
    binding.gqa_attn_set_wait_test(100_000)
    try:
        c.dense(ws)
    finally:
        binding.gqa_attn_set_wait_test(0)
    assert binding.gqa_attn_read_device_status(ws) & binding.GQA_DEV_WAIT_TIMEOUT
    binding.gqa_attn_clear_device_status(ws)
    o, status = c.dense(ws)
    assert status == 0
    parity.check(test_tree_gpu.f64(o), c.oracle()[0], "bf16")


@pytest.mark.parametrize("bs,D", [(64, 128), (64, 64), (16, 64)])
def test_copy_lost_piece_is_reported(bs, D):
    k, v = (inputs.randn((3, 40, 4, bs, D), s, torch.bfloat16, DEV) for s in (1, 2))
    k0, v0 = k.clone(), v.clone()
    src, dst = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in (np.arange(20), np.arange(20, 40)))
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    binding.gqa_attn_set_wait_test(100_000)
    try:
        binding.gqa_attn_copy_blocks(src, dst, None, k, v, ws)
        assert binding.gqa_attn_read_device_status(ws) & binding.GQA_DEV_WAIT_TIMEOUT
    finally:
        binding.gqa_attn_set_wait_test(0)
    # (what was written is what belongs there)
    for x, x0 in ((k, k0), (v, v0)):
        assert torch.equal(x[:, :20], x0[:, :20])
        assert ((x[:, 20:] == x0[:, 20:]) | (x[:, 20:] == x0[:, :20])).all()
    binding.gqa_attn_clear_device_status(ws)
    binding.gqa_attn_copy_blocks(src, dst, None, k, v, ws)
    assert binding.gqa_attn_read_device_status(ws) == 0
    assert torch.equal(k[:, 20:], k0[:, :20]) and torch.equal(v[:, 20:], v0[:, :20])
