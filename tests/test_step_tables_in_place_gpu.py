"""gqa_attn_step_tables with the lengths and the count over themselves, as a
running batch uses it, in each of its kernels: one block, a cluster of blocks
(more than 1,024 tokens), tokens in a grid of their own (more than 16,384), and
more than 1,024 requests.  Equal to the oracle step after step."""

import numpy as np
import pytest
import torch

import oracle
from gqa_attention_kv_decode_gb300 import binding
from test_step_tables_gpu import check, dev, draw

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


TOKENS = [1024, 1025, 2000, 8192, 16384, 16385, 40000]


@pytest.mark.parametrize("T", TOKENS)
@pytest.mark.parametrize("B", [1, 60, 1024, 1500])
@pytest.mark.parametrize("alias", [False, True])
def test_one_step(B, T, alias):
    bs, mb = 16, 80
    chunk = max(1, min(bs * mb, 2 * T // B))
    prior, new, table, stack, room = draw(B + T, B, bs, mb, chunk, room=T // bs + B)
    check(prior, new, T, bs, chunk, table, stack, room, alias=alias)


@pytest.mark.parametrize("T", TOKENS)
@pytest.mark.parametrize("B", [7, 1024])
def test_dense_cache(B, T):
    r = np.random.default_rng(B + T)
    cap = 3000
    rows = max(1, min(cap, 2 * T // B))
    new = np.where(r.random(B) < 0.2, -1, r.integers(0, rows + 1, B))
    check(r.integers(0, cap + 1, B), new, T, cap, rows, alias=True)


@pytest.mark.parametrize("T", [2000, 16384, 20000])
@pytest.mark.parametrize("B", [40, 1000])
def test_many_steps(B, T):
    """Requests that start, grow, finish and run out of blocks; every step in
    place, on what the step before left."""
    r = np.random.default_rng(T + B)
    bs, mb, chunk = 16, 40, max(2, T // B)
    pool = B * mb // 3
    prior, table = np.zeros(B, int), np.zeros((B, mb), int)
    stack, count = r.permutation(pool), pool
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    lens, table_t, stack_t, count_t, new_t = dev(prior), dev(table), dev(stack), dev([count]), dev(prior)
    out = {k: torch.empty(n, dtype=torch.int32, device=DEV)
           for k, n in {"q_starts": B + 1, "positions": T, "slots": T, "q_slots": T}.items()}
    seen = 0
    for step in range(12):
        new = np.where(r.random(B) < 0.6, r.integers(0, chunk + 1, B), 1)
        new[r.random(B) < 0.15] = -1
        new_t.copy_(dev(new))
        binding.gqa_attn_step_tables(lens, new_t, table_t, stack_t, count_t, lens, new_t, out["q_starts"],
                                     out["positions"], out["slots"], out["q_slots"], count_t, bs, chunk, ws)
        ref = oracle.step_tables(prior, new, T, bs, chunk, table, stack, count)
        seen |= ref["status"]
        assert binding.gqa_attn_read_device_status(ws) == seen  # (bits accumulate)
        prior, table, stack, count = ref["kv_lens"], ref["block_table"], ref["free_blocks"], int(ref["free_count"][0])
        for k, v in {**out, "kv_lens": lens, "q_lens": new_t, "block_table": table_t, "free_blocks": stack_t,
                     "free_count": count_t}.items():
            np.testing.assert_array_equal(v.cpu().numpy(), ref[k], err_msg=f"step {step}: {k}")
        held = [int(table[b, i]) for b in range(B) for i in range(-(-int(prior[b]) // bs))] + stack[:count].tolist()
        assert sorted(held) == list(range(pool))
