"""The oracle of the step tables against hand cases, and the host checks of
gqa_attn_step_tables (CPU)."""

import ctypes

import numpy as np
import pytest

import __graft_entry__
import oracle
from gqa_attention_kv_decode_gb300 import binding


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    return binding.lib()


def test_hand_case_grow_release_and_run_dry():
    # blocks of 4; stack [9, 8, 7], popped from the end; request 1 finishes and
    # gives back 5 and 6 first, so the pops are 6, 5, 7, 8, 9
    table = [[0, -7, -7], [5, 6, -7], [1, 2, -7], [3, -7, -7]]
    r = oracle.step_tables([4, 8, 7, 2], [5, -1, 2, 30], 40, 4, 40, table, [9, 8, 7, -7, -7, -7, -7, -7, -7, -7], 3)
    assert r["free_blocks"].tolist()[:5] == [9, 8, 7, 5, 6]
    # request 0: 4 + 5 rows, two new blocks; request 2: 7 + 2 rows, one;
    # request 3: 2 + 30 rows do not fit 3 blocks
    assert r["block_table"].tolist() == [[0, 6, 5], [5, 6, -7], [1, 2, 7], [3, -7, -7]]
    assert r["kv_lens"].tolist() == [9, 0, 9, 2] and r["q_lens"].tolist() == [5, 0, 2, 0]
    assert r["q_starts"].tolist() == [0, 5, 5, 7, 37] and r["free_count"].tolist() == [2]
    assert r["positions"].tolist()[:7] == [4, 5, 6, 7, 8, 7, 8]
    assert r["slots"].tolist()[:7] == [24, 25, 26, 27, 20, 11, 28]
    assert r["q_slots"].tolist()[:7] == [0, 1, 2, 3, 4, 80, 81]
    assert (r["slots"][7:] == -1).all() and (r["positions"][7:] == 0).all()
    assert r["status"] == 1


def test_hand_case_out_of_blocks_is_all_or_nothing():
    # three free blocks; request 0 takes two, request 1 needs two (refused),
    # request 2 none (served), request 3 one (refused: it comes after)
    table = np.zeros((4, 3), dtype=int)
    r = oracle.step_tables([0, 0, 1, 0], [8, 5, 1, 1], 16, 4, 8, table, [1, 2, 3, 0], 3)
    assert r["q_lens"].tolist() == [8, 0, 1, 0] and r["kv_lens"].tolist() == [8, 0, 2, 0]
    assert r["free_count"].tolist() == [1] and r["block_table"][0].tolist() == [3, 2, 0]
    assert r["slots"][8:13].tolist() == [-1] * 5 and r["slots"][13] == 1 and r["slots"][14] == -1
    assert r["status"] == 16


def test_hand_case_dense():
    r = oracle.step_tables([3, 10, 0], [2, 1, 0], 4, 10, 2)
    assert r["slots"].tolist() == [3, 4, -1, -1] and r["q_slots"].tolist() == [0, 1, -1, -1]
    assert r["kv_lens"].tolist() == [5, 10, 0] and r["status"] == 1


P = ctypes.c_void_p(256)  # never dereferenced: shape checks come first


@pytest.mark.parametrize("bad", [
    dict(B=0), dict(B=65536), dict(T=0), dict(bs=0), dict(nb=0), dict(mb=0), dict(q_rows=0),
    dict(B=65535, q_rows=40000), dict(B=65535, mb=40000, bs=1), dict(nb=1 << 20, bs=1 << 12),
    dict(mb=1 << 20, bs=1 << 12, nb=1),
])
def test_sizes_are_checked_on_the_host(lib, bad):
    a = dict(B=2, T=4, bs=64, nb=8, mb=4, q_rows=2) | bad
    rc = lib.gqa_attn_step_tables(*[P] * 12, a["B"], a["T"], a["bs"], a["nb"], a["mb"], a["q_rows"], P, 256, None)
    assert rc == binding.GQA_ERR_INVALID_ARG


def test_a_dense_cache_takes_no_stack(lib):
    rc = lib.gqa_attn_step_tables(P, P, None, P, None, P, P, P, P, P, P, None, 2, 4, 64, 0, 0, 2, P, 256, None)
    assert rc == binding.GQA_ERR_INVALID_ARG
