"""The oracle of drafted tokens and shared pages against hand cases, and the host
checks of their entry points (CPU)."""

import ctypes

import numpy as np
import pytest
import torch

import __graft_entry__
import oracle
from gqa_attention_kv_decode_gb300 import binding


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    return binding.lib()


# ---------------------------------------------------------------- the oracle by hand

def test_tree_tables_by_hand():
    #   0 - 1 - 3
    #     \ 2      4 (a root of its own)
    parents = [[-1, 0, 0, 1, -1]]
    mask, pos, status = oracle.tree_tables(parents, [5], None, np.zeros((1, 5, 1)), [25], [2], np.zeros(8))
    assert mask[0, :, 0].tolist() == [1, 3, 5, 11, 16] and status == 0
    assert pos.tolist() == [0, 0, 20, 21, 21, 22, 20, 0]
    # the last two nodes are the queries
    mask, pos, status = oracle.tree_tables(parents, [5], [2], np.full((1, 2, 1), 7), [25], [0], np.zeros(2))
    assert mask[0, :, 0].tolist() == [11, 16] and pos.tolist() == [22, 20] and status == 0


def test_tree_tables_bad_parents_and_lengths():
    mask, _, status = oracle.tree_tables([[0, 5, -2, 2]], [4], None, np.zeros((1, 4, 1)))
    assert mask[0, :, 0].tolist() == [1, 2, 4, 12] and status == 128
    mask, _, status = oracle.tree_tables([[-1, 0]], [3], [-1], np.full((1, 2, 1), 9))
    assert (mask == 9).all() and status == 1


def test_attention_tree_is_attention_of_the_visible_rows():
    r = np.random.default_rng(0)
    q, k, v = r.standard_normal((1, 4, 3, 8)), r.standard_normal((1, 2, 9, 8)), r.standard_normal((1, 2, 9, 8))
    mask = np.array([[[1], [3], [0]]], dtype=np.int32)
    o, status = oracle.attention_tree(q, k, v, mask, [3], [3], [9], 0.3, np.zeros_like(q))
    assert status == 0
    for h in range(4):
        for i, rows in enumerate(([0, 1, 2, 3, 4, 5, 6], [0, 1, 2, 3, 4, 5, 6, 7], [0, 1, 2, 3, 4, 5])):
            ref = oracle.attention(q[:, h:h + 1, i:i + 1], k[:, h // 2:h // 2 + 1, rows], v[:, h // 2:h // 2 + 1, rows],
                                   scale=0.3)["o"]
            np.testing.assert_allclose(o[0, h, i], ref[0, 0, 0], rtol=1e-12)
    chain, _ = oracle.attention_tree(q, k, v, None, None, None, [9], 0.3, np.zeros_like(q))
    np.testing.assert_allclose(chain, oracle.attention(q, k, v, scale=0.3, causal=True)["o"], rtol=1e-12)


def test_attention_tree_of_rows_that_see_nothing():
    one = np.ones((1, 1, 2, 4))
    o, status = oracle.attention_tree(one, one, one, np.zeros((1, 2, 1), np.int32), None, None, [2], 1.0, one * 5)
    assert status == 2 and not o.any()


def test_compact_rows_by_hand():
    k = np.arange(8.0).reshape(1, 4, 1, 2, 1)
    table = [[3, 1, 0]]  # rows: 6 7 2 3 0 1
    kk, vv, lens, status = oracle.compact_rows([[0, 2, 3]], [3], [4], [5], table, k, k + 10)
    # base 1: node 0 is 7, 1 is 2, 2 is 3, 3 is 0
    assert lens.tolist() == [4] and status == 0
    assert kk[0, :, 0, :, 0].tolist() == [[0, 1], [3, 0], [4, 5], [6, 7]]
    assert (vv == kk + 10).all()
    for path in ([0, 0, 1], [1, 0, 2], [0, 1, 4], [-1, 0, 1]):
        kk, _, lens, status = oracle.compact_rows([path], [3], [4], [5], table, k, k)
        assert status == 128 and lens.tolist() == [1] and (kk == k).all()


def test_fork_tables_by_hand():
    table = np.array([[4, 5, 6], [4, 7, 0], [8, 0, 0]])
    shared = np.zeros(10, int)
    shared[4] = 1
    none = np.full((4, 3), -9)
    # two continue request 0 (the second keeps more, and so owns block 6), one keeps a
    # part of the shared block of request 1, request 2 ends
    out = oracle.fork_tables([0, 0, 1, -1], [9, 10, 2, 0], [10, 7, 3], table, shared, [1, 2, 3] + [0] * 7, 3, none, 4)
    assert out["status"] == 0
    assert out["block_table"].tolist() == [[4, 5, 3], [4, 5, 6], [2, -9, -9], [-9, -9, -9]]
    assert out["kv_lens"].tolist() == [9, 10, 2, 0]
    assert [out[x].tolist() for x in ("copy_src", "copy_dst", "copy_rows")] == [[6, -1, 4, -1], [3, -1, 2, -1], [1, 0, 2, 0]]
    # block 4 loses request 1 and gains request 0's fork, 5 is shared by both
    assert out["shared"].tolist() == [0, 0, 0, 0, 1, 1, 0, 0, 0, 0]
    assert out["free_count"].tolist() == [3] and out["free_blocks"][:3].tolist() == [1, 7, 8]


def test_fork_tables_without_free_blocks():
    out = oracle.fork_tables([0, 0], None, [6], [[2, 3]], [0] * 4, [0] * 4, 0, np.zeros((2, 2)), 4)
    assert out["status"] == 16 and out["kv_lens"].tolist() == [6, 4] and out["shared"].tolist() == [0, 0, 1, 0]


def test_copy_blocks_by_hand():
    k = np.arange(6.0).reshape(1, 3, 1, 2, 1)
    kk, vv, status = oracle.copy_blocks([0, -1, 0], [2, 1, 1], [1, 2, 5], k, k)
    assert kk.reshape(3, 2).tolist() == [[0, 1], [0, 1], [0, 5]] and status == 1 and (vv == kk).all()
    kk, _, status = oracle.copy_blocks([3, 0], [0, -1], None, k, k)
    assert status == 8 and (kk == k).all()


# ---------------------------------------------------------------- host checks

P = ctypes.c_void_p(256)  # never dereferenced: shape checks come first
INVALID = binding.GQA_ERR_INVALID_ARG


def tree(lib, paged, **change):
    a = dict(B=2, Hq=8, Hkv=2, D=64, Tq=4, W=1, S=64, L=64, scale=0.125, dtype=1, nb=4, mb=2, mask=P, tl=P, table=P) | change
    if paged:
        return lib.gqa_attn_decode_tree_paged(P, P, P, a["table"], a["mask"], P, a["tl"], P, P, a["B"], a["Hq"],
                                              a["Hkv"], a["D"], a["Tq"], a["W"], a["S"], a["nb"], a["mb"], a["L"],
                                              a["scale"], a["dtype"], P, 1 << 30, None)
    return lib.gqa_attn_decode_tree(P, P, P, a["mask"], P, a["tl"], P, P, a["B"], a["Hq"], a["Hkv"], a["D"], a["Tq"],
                                    a["W"], a["S"], a["L"], a["scale"], a["dtype"], P, 1 << 30, None)


@pytest.mark.parametrize("bad", [
    dict(B=0), dict(B=65536), dict(Hq=0), dict(Hkv=0), dict(Hq=7), dict(D=96), dict(Tq=0), dict(Tq=1025), dict(L=0),
    dict(L=65), dict(S=0), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
    dict(B=60000, Hq=64, Hkv=64, Tq=1024),
])
def test_tree_shapes_are_checked_on_the_host(lib, bad):
    assert tree(lib, False, **bad) == INVALID
    if "L" not in bad and "S" not in bad:
        assert tree(lib, True, **bad) == INVALID


@pytest.mark.parametrize("bad", [dict(S=0), dict(nb=0), dict(mb=0), dict(L=129), dict(nb=1 << 24), dict(table=None)])
def test_pools_are_checked_on_the_host(lib, bad):
    assert tree(lib, True, **bad) == INVALID


def test_workspace_size_of_a_bad_shape_is_zero(lib):
    size = binding.gqa_attn_decode_tree_workspace_size
    assert size(2, 8, 2, 64, 4, 100) >= 256
    for bad in ((0, 8, 2, 64, 4, 100), (2, 7, 2, 64, 4, 100), (2, 8, 2, 80, 4, 100), (2, 8, 2, 64, 0, 100),
                (2, 8, 2, 64, 1025, 100), (2, 8, 2, 64, 4, 0)):
        assert size(*bad) == 0


def tables(lib, **change):
    a = dict(B=2, N=40, Tq=8, W=2, T=16, kv=P, st=P, pos=P) | change
    return lib.gqa_attn_tree_tables(P, P, P, a["kv"], a["st"], P, a["pos"], a["B"], a["N"], a["Tq"], a["W"], a["T"], P,
                                    256, None)


@pytest.mark.parametrize("bad", [
    dict(B=0), dict(B=65536), dict(N=0), dict(N=1025, W=33), dict(Tq=0), dict(Tq=1025), dict(W=1), dict(W=3), dict(T=0),
    dict(kv=None), dict(st=None), dict(pos=None), dict(kv=None, st=None),
])
def test_tree_tables_are_checked_on_the_host(lib, bad):
    assert tables(lib, **bad) == INVALID


def compact(lib, **change):
    a = dict(table=P, NL=2, B=3, P=5, Hkv=2, D=64, bs=16, nb=9, mb=4, dtype=1) | change
    return lib.gqa_attn_compact_rows(P, P, P, P, a["table"], P, P, P, a["NL"], a["B"], a["P"], a["Hkv"], a["D"], a["bs"],
                                     a["nb"], a["mb"], a["dtype"], P, 256, None)


@pytest.mark.parametrize("bad", [
    dict(B=0), dict(B=65536), dict(P=0), dict(P=1025), dict(NL=0), dict(Hkv=0), dict(D=32), dict(bs=0), dict(nb=0),
    dict(mb=0), dict(dtype=2), dict(NL=1 << 20), dict(nb=1 << 26), dict(table=None), dict(mb=1 << 28),
])
def test_compact_is_checked_on_the_host(lib, bad):
    assert compact(lib, **bad) == INVALID


FORK = ("src", "keep", "held", "table", "shared", "stack", "count", "out", "kv", "shared_out", "stack_out", "count_out",
        "csrc", "cdst", "crows")
AT = {name: ctypes.c_void_p(256 * (i + 2)) for i, name in enumerate(FORK)}
REACHES_THE_DEVICE = (binding.GQA_ERR_CUDA, binding.GQA_ERR_NOT_DEVICE_PTR)  # (without one, and with these pointers)


def fork(lib, **change):
    a = dict(B_in=3, B=4, mb=5, bs=16, nb=20) | AT | change
    return lib.gqa_attn_fork_tables(*(a[x] for x in FORK), a["B_in"], a["B"], a["mb"], a["bs"], a["nb"], P, 256, None)


def test_fork_arrays_that_may_not_be_one(lib):
    for now, before in (("shared_out", "shared"), ("stack_out", "stack"), ("count_out", "count")):
        assert fork(lib, **{now: AT[before]}) in REACHES_THE_DEVICE
    assert fork(lib, keep=None) in REACHES_THE_DEVICE
    for now, before in (("out", "table"), ("kv", "held"), ("kv", "keep"), ("kv", "src"), ("csrc", "src"), ("cdst", "csrc"),
                        ("crows", "keep"), ("shared_out", "stack_out"), ("count_out", "kv"), ("out", "stack"), ("crows", "count"),
                        ("stack_out", "table")):
        assert fork(lib, **{now: AT[before]}) == INVALID


@pytest.mark.parametrize("bad", [
    dict(B=0), dict(B=8193), dict(B_in=0), dict(B_in=8193), dict(mb=0), dict(bs=0), dict(nb=0),
    dict(B=8192, mb=1 << 17, bs=1), dict(mb=1 << 20, bs=1 << 12), dict(nb=1 << 28),
])
def test_fork_is_checked_on_the_host(lib, bad):
    assert fork(lib, **bad) == INVALID


def copy(lib, **change):
    a = dict(NL=2, n=3, Hkv=2, D=64, bs=16, nb=9, dtype=1) | change
    return lib.gqa_attn_copy_blocks(P, P, P, P, P, a["NL"], a["n"], a["Hkv"], a["D"], a["bs"], a["nb"], a["dtype"], P, 256,
                                    None)


@pytest.mark.parametrize("bad", [dict(n=0), dict(n=65536), dict(NL=0), dict(Hkv=0), dict(D=256), dict(bs=0), dict(nb=0),
                                 dict(dtype=-1), dict(NL=1 << 20), dict(nb=1 << 27)])
def test_copy_is_checked_on_the_host(lib, bad):
    assert copy(lib, **bad) == INVALID


# ---------------------------------------------------------------- what the binding refuses (CPU tensors)

def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def cache(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


WS = torch.zeros(256, dtype=torch.uint8)


@pytest.mark.parametrize("change,error", [
    (dict(q=cache(2, 8, 64)), ValueError), (dict(k=cache(3, 2, 32, 64)), ValueError), (dict(v=cache(2, 2, 31, 64)), ValueError),
    (dict(o=cache(2, 8, 3, 64)), ValueError), (dict(v=cache(2, 2, 32, 64, dtype=torch.float16)), TypeError),
    (dict(mask=i32(2, 4)), ValueError), (dict(mask=i32(2, 3, 1)), ValueError), (dict(mask=i32(2, 4, 1).long()), TypeError),
    (dict(ql=i32(3)), ValueError), (dict(tl=i32(1)), ValueError), (dict(kl=i32(2).long()), TypeError), (dict(kl=None), TypeError),
    (dict(k=cache(2, 2, 64, 32).transpose(2, 3)), ValueError), (dict(ws=None), TypeError),
])
def test_tree_tensors_are_checked(lib, change, error):
    a = dict(q=cache(2, 8, 4, 64), k=cache(2, 2, 32, 64), v=cache(2, 2, 32, 64), mask=i32(2, 4, 1), ql=i32(2), tl=i32(2),
             kl=i32(2), o=cache(2, 8, 4, 64), ws=WS) | change
    with pytest.raises(error):
        binding.gqa_attn_decode_tree(a["q"], a["k"], a["v"], a["mask"], a["ql"], a["tl"], a["kl"], a["o"], 0.1, a["ws"], stream=0)


def test_cache_tensors_are_checked(lib):
    k = cache(2, 9, 2, 16, 64)
    for kc, vc, error in ((k, k[0], ValueError), (k[0, 0], k[0, 0], ValueError), (k, k.float(), TypeError), (k.half(), k.half(), TypeError),
                          (k.transpose(0, 1), k.transpose(0, 1), ValueError)):
        with pytest.raises(error):
            binding.gqa_attn_copy_blocks(i32(3), i32(3), None, kc, vc, WS, stream=0)
        with pytest.raises(error):
            binding.gqa_attn_compact_rows(i32(2, 3), i32(2), i32(2), i32(2), i32(2, 2), kc, vc, i32(2), WS, stream=0)
    with pytest.raises(ValueError):
        binding.gqa_attn_copy_blocks(i32(3), i32(2), None, k, k, WS, stream=0)
    with pytest.raises(ValueError):
        binding.gqa_attn_compact_rows(i32(2, 3), i32(2), i32(2), i32(2), i32(3, 2), k, k, i32(2), WS, stream=0)
