"""The shared-prefix oracle against hand values and invariants, and the host
checks of the shared-prefix entry points (CPU)."""

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


def draws(B, Hq, Hkv, D, P, S, seed=0):
    r = np.random.default_rng(seed)
    f = r.standard_normal
    return f((B, Hq, 1, D)), f((Hkv, P, D)), f((Hkv, P, D)), f((B, Hkv, S, D)), f((B, Hkv, S, D))


def test_equals_attention_on_copied_prefixes():
    q, kp, vp, k, v = draws(3, 6, 2, 8, 5, 4)
    lens = [4, 0, 2]
    kk = np.concatenate([np.broadcast_to(kp, (3, *kp.shape)), k], 2)
    vv = np.concatenate([np.broadcast_to(vp, (3, *vp.shape)), v], 2)
    ref = oracle.attention(q, kk, vv, kv_lens=np.array(lens) + 5, scale=0.3)["o"]
    np.testing.assert_allclose(oracle.attention_shared_prefix(q, kp, vp, k, v, lens, 0.3), ref, rtol=1e-13, atol=1e-15)


def test_one_visible_row_is_its_value_and_none_is_zeros():
    q, kp, vp, k, v = draws(2, 4, 2, 8, 1, 3)
    o = oracle.attention_shared_prefix(q, kp, vp, k, v, [0, 0], 0.5)
    for h in range(4):
        np.testing.assert_allclose(o[:, h, 0], np.broadcast_to(vp[h // 2, 0], (2, 8)), rtol=1e-14)
    o = oracle.attention_shared_prefix(q, kp[:, :0], vp[:, :0], k, v, [0, 1], 0.5)
    assert (o[0] == 0).all()
    np.testing.assert_allclose(o[1, 3, 0], v[1, 1, 0], rtol=1e-14)


P = ctypes.c_void_p(256)  # never dereferenced: shape checks come first
GOOD = dict(B=2, Hq=8, Hkv=2, D=64, P_cap=100, maxp=100, S=50, L=50, scale=0.1, dtype=1)


@pytest.mark.parametrize("bad,rc", [
    (dict(B=0), -1), (dict(B=65536), -1), (dict(Hkv=3), -1), (dict(D=96), -1), (dict(maxp=0), -1), (dict(maxp=101), -1),
    (dict(L=0), -1), (dict(L=51), -1), (dict(scale=0.0), -1), (dict(scale=float("inf")), -1), (dict(dtype=5), -1),
    (dict(P_cap=2 ** 31 - 1, maxp=2 ** 31 - 1), -1), (dict(B=65535, Hq=128, Hkv=64), -1),
    (dict(dtype=0), -2), (dict(Hq=258, Hkv=2), -2),
])
def test_dense_arguments_are_checked_on_the_host(lib, bad, rc):
    a = GOOD | bad
    got = lib.gqa_attn_decode_shared_prefix(P, P, P, P, P, P, P, P, a["B"], a["Hq"], a["Hkv"], a["D"], a["P_cap"],
                                            a["maxp"], a["S"], a["L"], a["scale"], a["dtype"], P, 1 << 30, None)
    assert got == rc


GOODP = dict(B=2, Hq=8, Hkv=2, D=64, bs=64, nb=20, mpb=4, mb=3, maxp=256, L=192, scale=0.1, dtype=1)


@pytest.mark.parametrize("bad,rc", [
    (dict(bs=0), -1), (dict(nb=0), -1), (dict(mpb=0), -1), (dict(mb=0), -1), (dict(maxp=257), -1), (dict(L=193), -1),
    (dict(maxp=0), -1), (dict(nb=1 << 24, bs=1 << 10, maxp=1, L=1), -1), (dict(bs=32, maxp=1, L=1), -2),
    (dict(bs=96, maxp=1, L=1), -2), (dict(dtype=0), -2), (dict(Hq=258, Hkv=2), -2),
])
def test_paged_arguments_are_checked_on_the_host(lib, bad, rc):
    a = GOODP | bad
    got = lib.gqa_attn_decode_shared_prefix_paged(P, P, P, P, P, P, P, P, a["B"], a["Hq"], a["Hkv"], a["D"], a["bs"],
                                                  a["nb"], a["mpb"], a["mb"], a["maxp"], a["L"], a["scale"],
                                                  a["dtype"], P, 1 << 30, None)
    assert got == rc


def test_workspace_size_is_zero_for_shapes_the_calls_refuse(lib):
    size = binding.gqa_attn_decode_shared_prefix_workspace_size
    assert size(2, 8, 2, 64, 100, 50) > 0
    for bad in ((2, 8, 3, 64, 100, 50), (2, 8, 2, 96, 100, 50), (2, 8, 2, 64, 0, 50), (2, 8, 2, 64, 100, 0),
                (2, 258, 2, 64, 100, 50)):
        assert size(*bad) == 0
