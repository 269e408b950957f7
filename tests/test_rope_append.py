"""The oracle of the norm-rotate-append against hand cases and invariants, the
angle-table helper, and the host checks of gqa_attn_rope_append (CPU)."""

import ctypes
import math

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


def test_rms_norm_by_hand():
    # mean square 12.5 + eps 3.5 = 16
    y = oracle.rms_norm([[3.0, 4.0]], [2.0, 0.5], 3.5)
    np.testing.assert_allclose(y, [[1.5, 0.5]], rtol=1e-15)


@pytest.mark.parametrize("adjacent", [False, True])
def test_rotation_by_hand(adjacent):
    """A quarter turn of the first pair, half a turn of the second; dims past
    the rotated ones stay."""
    x = np.array([[[1.0, 2.0, 3.0, 4.0, 5.0, 6.0]]])
    cos, sin = np.array([[0.0, -1.0]]), np.array([[1.0, 0.0]])
    y = oracle.rotate(x, cos, sin, adjacent)
    want = [-2.0, 1.0, -3.0, -4.0, 5.0, 6.0] if adjacent else [-3.0, -2.0, 1.0, -4.0, 5.0, 6.0]
    np.testing.assert_array_equal(y[0, 0], want)


def test_rotated_scores_depend_on_the_distance_only():
    r = np.random.default_rng(0)
    q, k = r.standard_normal((1, 1, 64)), r.standard_normal((1, 1, 64))
    t = binding.rope_table(300, 64, device="cpu").double().numpy()
    s = []
    for m, n in ((10, 3), (207, 200), (299, 292)):
        a = oracle.rotate(q, t[m:m + 1, :32], t[m:m + 1, 32:], False)
        b = oracle.rotate(k, t[n:n + 1, :32], t[n:n + 1, 32:], False)
        s.append(float((a * b).sum()))
    # every table entry is off by at most 2^-25, so each of the 64 terms of a
    # score by about 4 * 2^-25 * |q_i k_i|
    assert max(s) - min(s) <= 2 * 64 * 4 * 2.0 ** -25 * 9


def test_rope_table_values():
    t = binding.rope_table(200001, 128, base=1e6, device="cpu")
    assert t.shape == (200001, 128) and t.dtype == torch.float32
    for pos in (0, 1, 4097, 200000):
        for i in (0, 1, 63):
            a = pos * 1e6 ** (-2 * i / 128)
            # the angle in 64 bits: off by a few 2^-53 of it; the entry by half an fp32 step
            tol = 2.0 ** -25 + 8 * a * 2.0 ** -53
            assert abs(float(t[pos, i]) - math.cos(a)) <= tol
            assert abs(float(t[pos, 64 + i]) - math.sin(a)) <= tol


def test_append_places_rows_by_hand():
    q = np.arange(2 * 1 * 2).reshape(2, 1, 2) + 1.0
    k, v = q * 10, q * 100
    z = np.zeros((2, 1, 3, 2))
    qo, kc, vc, status = oracle.rope_append(q, k, v, None, None, 0.0, None, None, [4, -1], [-1, 0], z, z, z, False)
    assert status == 0
    assert qo[0, 0, 0].tolist() == [3.0, 4.0] and np.count_nonzero(qo) == 2
    assert kc[1, 0, 1].tolist() == [10.0, 20.0] and np.count_nonzero(kc) == 2
    assert vc[1, 0, 1].tolist() == [100.0, 200.0] and np.count_nonzero(vc) == 2


P = ctypes.c_void_p(256)  # never dereferenced: shape checks come first

GOOD = dict(qs=256, ks=128, vs=128, eps=1e-6, T=3, Hq=4, Hkv=2, D=64, rot=64, max_pos=9, adjacent=0, nb=2, bs=4, qg=3,
            qr=1, dtype=1, cs=P, pos=P, q_slots=P)


def call(lib, **change):
    a = GOOD | change
    return lib.gqa_attn_rope_append(P, P, P, a["qs"], a["ks"], a["vs"], P, P, a["eps"], a["cs"], a["pos"], P,
                                    a["q_slots"], P, P, P, a["T"], a["Hq"], a["Hkv"], a["D"], a["rot"], a["max_pos"],
                                    a["adjacent"], a["nb"], a["bs"], a["qg"], a["qr"], a["dtype"], P, 256, None)


@pytest.mark.parametrize("bad", [
    dict(T=0), dict(Hq=0), dict(Hkv=0), dict(Hq=3), dict(D=96), dict(dtype=2), dict(rot=8), dict(rot=80),
    dict(rot=-16), dict(max_pos=0), dict(adjacent=2), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
    dict(nb=0), dict(bs=0), dict(qg=0), dict(qr=0), dict(nb=1 << 20, bs=1 << 12), dict(qg=1 << 20, qr=1 << 12),
    dict(q_slots=None, T=4), dict(T=1 << 28), dict(qs=248), dict(ks=120), dict(vs=120), dict(qs=260), dict(ks=132), dict(vs=132),
    dict(rot=0), dict(rot=0, cs=None), dict(rot=0, pos=None),
])
def test_arguments_are_checked_on_the_host(lib, bad):
    assert call(lib, **bad) == binding.GQA_ERR_INVALID_ARG
