"""Shared-prefix decode of more than 1,024 requests, whose own rows the decode
kernel takes: own rows of one split and of several, against the fp64 oracle."""

import numpy as np
import pytest
import torch

import oracle
import parity
from gqa_attention_kv_decode_gb300 import binding, inputs

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def f64(t):
    return t.detach().float().cpu().numpy()


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("B,Hq,Hkv,D,S,P", [(1025, 2, 1, 64, 3000, 200), (1100, 8, 1, 128, 2100, 129),
                                            (1025, 4, 2, 64, 1024, 1), (1300, 17, 1, 64, 1025, 700)])
@pytest.mark.parametrize("paged", [False, True])
def test_several_splits_of_own_rows(B, Hq, Hkv, D, S, P, paged):
    lens = np.random.default_rng(S).integers(0, S + 1, B)
    special = [0, 1, 63, 64, 65, 1023, 1024, min(1025, S), S - 1, S]
    lens[:len(special)] = special
    if not paged:  # (more than one split is what is asked for, in the larger shapes)
        n_split, _, _ = binding.gqa_attn_decode_plan_for(B, Hq, Hkv, D, S, binding.GQA_BF16, 152, binding.GQA_PLAN_DECODE)
        assert n_split == -(-S // 1024)
    q = inputs.randn((B, Hq, 1, D), 61, BF16, DEV)
    kp, vp = (inputs.randn((Hkv, P + 3, D), s, BF16, DEV) for s in (62, 63))
    kp[:, P:], vp[:, P:] = float("nan"), float("nan")
    g = torch.Generator(device=DEV).manual_seed(64)
    bs = 64
    n_own, n_pre = -(-S // bs), -(-P // bs)
    ws = binding.decode_shared_prefix_workspace(B, Hq, Hkv, D, P + 3, S)
    ws[256:] = 0xFF
    if paged:  # every request has a stretch of one pool, from a block of its own on
        n = 200 + n_own + n_pre
        kpool, vpool = (torch.randn((n, Hkv, bs, D), generator=g, device=DEV).to(BF16) for _ in range(2))
        for pool, x in ((kpool, kp), (vpool, vp)):
            pool[:n_pre] = torch.cat([x[:, :P], x.new_zeros((Hkv, n_pre * bs - P, D))], 1).unflatten(
                1, (n_pre, bs)).transpose(0, 1)
        table = n_pre + (np.arange(B) * 7 % 200)[:, None] + np.arange(n_own)[None]
        o = binding.decode_shared_prefix_paged(q, kpool, vpool, i32(np.arange(n_pre)), i32(table), i32(lens), P, S,
                                               prefix_len=i32([P]), workspace=ws)
        own = lambda pool, b: f64(pool[table[b]].transpose(0, 1).reshape(Hkv, n_own * bs, D)[:, :S])  # noqa: E731
        ko, vo = kpool, vpool
    else:
        ko, vo = (torch.randn((B, Hkv, S, D), generator=g, device=DEV).to(BF16) for _ in range(2))
        for t in (ko, vo):
            inputs.poison_tail(t, [int(x) for x in lens])
        o = binding.decode_shared_prefix(q, kp, vp, ko, vo, prefix_len=i32([P]), kv_lens=i32(lens), max_prefix_len=P,
                                         workspace=ws)
        own = lambda t, b: np.nan_to_num(f64(t[b]))  # noqa: E731
    assert binding.gqa_attn_read_device_status(ws) == 0
    some = sorted({*range(len(special)), *range(11, B, 37), B - 1})
    ref = oracle.attention_shared_prefix(f64(q)[some], f64(kp)[:, :P], f64(vp)[:, :P], np.stack([own(ko, b) for b in some]),
                                         np.stack([own(vo, b) for b in some]), lens[some], D ** -0.5)
    parity.check(f64(o)[some], ref, "bf16")
    assert o.isfinite().all()
