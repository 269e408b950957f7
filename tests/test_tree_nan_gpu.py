"""NaN and infinities in rows that are seen (attention of drafted rows): a row with a NaN
or a +inf among its scores is NaN, however the call shares out the keys, a -inf score has
no weight, and the other rows are as they were."""

import numpy as np
import pytest
import torch

import oracle
import parity
from gqa_attention_kv_decode_gb300 import binding
from test_tree_gpu import Case, f64

pytestmark = pytest.mark.gpu
PLANS = (0, 1, 2, 4, 8)  # as planned, as one list, in clusters
# (one row tile and a pair, each with D = 64 and 128; keys of each request: of one tile, and of several)
SHAPES = [(8, 2, 64, 9), (8, 2, 128, 9), (8, 1, 64, 25), (8, 1, 128, 25)]
LENS = [[128, 30], [128 * 2 + 9, 300], [128 * 7 + 25, 1025]]


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def check(c, nan, status=0):
    """nan: bool [B, Hq, Tq], the rows that are NaN in every column."""
    ref, _ = c.oracle()
    for plan in PLANS:
        with binding.plan_override(prefill_kv_split=plan):
            # (a bound above one tile, so that a unit may be shared by several CTAs)
            o, seen = c.dense()
        o = f64(o)
        assert (np.isnan(o) == nan[..., None]).all(), f"plan {plan}: rows that are NaN"
        parity.check(np.where(nan[..., None], 0.0, o), np.where(nan[..., None], 0.0, ref), "bf16", f"plan {plan}")
        assert seen == status, f"plan {plan}"


def case(Hq, Hkv, D, Tq, lens, seed=0):
    lens = [max(Tq, n) for n in lens]
    return Case(len(lens), Hq, Hkv, D, Tq, lens, S=max(lens) + 130, mask="tree", seed=seed)


@pytest.mark.parametrize("Hq,Hkv,D,Tq", SHAPES)
@pytest.mark.parametrize("lens", LENS)
def test_a_query_with_a_nan(Hq, Hkv, D, Tq, lens):
    c = case(Hq, Hkv, D, Tq, lens)
    nan = np.zeros(c.q.shape[:3], bool)
    for b, h, i in ((0, 1, 3), (1, Hq - 1, Tq - 1), (1, 0, 0)):
        c.q[b, h, i, 7] = float("nan")
        nan[b, h, i] = True
    check(c, nan)


@pytest.mark.parametrize("Hq,Hkv,D,Tq", SHAPES)
@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("alone", [False, True])
def test_a_drafted_key_with_a_nan(Hq, Hkv, D, Tq, lens, alone):
    """The queries that see it are NaN; `alone`: each query sees no other drafted row, so that a tile may
    have nothing but the NaN for its row."""
    c = case(Hq, Hkv, D, Tq, lens, 1)
    if alone:
        c.mask[:] = 0
        for i in range(Tq):
            c.mask[:, i, i // 32] = np.uint32(1 << i % 32).astype(np.int32)
        c.k = torch.nan_to_num(c.k)
    nan = np.zeros(c.q.shape[:3], bool)
    for b, node in ((0, 2), (1, Tq - 1)):
        c.k[b, :, c.kv_lens[b] - Tq + node, 1] = float("nan")
        nan[b] |= oracle.tree_visible(c.mask[b], Tq, Tq, Tq, c.kv_lens[b])[:, c.kv_lens[b] - Tq + node]
    assert nan.any() and not nan.all()
    check(c, nan)


@pytest.mark.parametrize("Hq,Hkv,D,Tq", SHAPES)
@pytest.mark.parametrize("lens", LENS[1:])
def test_infinite_keys(Hq, Hkv, D, Tq, lens):
    """A key with an infinity that every query sees: rows with a score of +inf are NaN, as inf - inf is;
    for those with -inf the key has no weight."""
    c = case(Hq, Hkv, D, Tq, lens, 2)
    nan = np.zeros(c.q.shape[:3], bool)
    for b, row, value in ((0, 5, float("inf")), (1, 140, float("-inf"))):
        c.k[b, :, row, 3] = value
        nan[b] |= f64(c.q)[b, :, :, 3] * value > 0
    assert nan.any() and not nan.all()
    q, k, v = f64(c.q), np.nan_to_num(f64(c.k), nan=0.0, posinf=np.inf, neginf=-np.inf), np.nan_to_num(f64(c.v))
    with np.errstate(all="ignore"):
        want = oracle.attention_tree(q, k, v, c.mask, None, None, c.kv_lens, c.scale, np.full(c.q.shape, 3.0))
    c.oracle = lambda: want
    check(c, nan)


@pytest.mark.parametrize("Hq,Hkv,D,Tq", SHAPES)
def test_infinite_values(Hq, Hkv, D, Tq):
    """An infinity in a row of V that all queries see is that column's."""
    c = case(Hq, Hkv, D, Tq, LENS[1], 3)
    c.v[0, :, 100, 4] = float("inf")
    ref = f64(c.dense()[0])
    ref[0, :, :, 4] = 0
    assert np.isfinite(ref).all()
    for plan in PLANS:
        with binding.plan_override(prefill_kv_split=plan):
            o, seen = c.dense()
        o = f64(o)
        assert (o[0, :, :, 4] == np.inf).all() and seen == 0
        o[0, :, :, 4] = 0
        parity.check(o, ref, "bf16", f"plan {plan}")
