"""The lost-copy path of the drafted rows' attention (see test_tree_wait_gpu.py) in each of its
kernels: the list of all units and clusters of CTAs, one row tile and a pair, D = 64 and 128."""

import numpy as np
import pytest

import parity
from gqa_attention_kv_decode_gb300 import binding
from test_tree_gpu import Case, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Tq", [5, 50])  # two slots of their own, and a pair of row tiles
@pytest.mark.parametrize("plan", [1, 2, 8])
def test_a_lost_copy_is_reported_by_every_kernel(D, Tq, plan):
    c = Case(3, 16, 4, D, Tq, [3000, 700, 90])
    ws = c.workspace()
    with binding.plan_override(prefill_kv_split=plan):
        binding.gqa_attn_set_wait_test(100_000)
        try:
            lost, status = c.dense(ws)
        finally:
            binding.gqa_attn_set_wait_test(0)
        assert status & binding.GQA_DEV_WAIT_TIMEOUT
        if plan > 1:  # a cluster's rows of lost tiles are NaN, not what is left without these tiles
            assert np.isnan(f64(lost)).all()
            assert not status & binding.GQA_DEV_EMPTY_REQUEST
        binding.gqa_attn_clear_device_status(ws)
        o, status = c.dense(ws)
    assert status == 0
    parity.check(f64(o), c.oracle()[0], "bf16")
