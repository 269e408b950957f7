"""Lengths of a shared-prefix decode that have to be clamped are reported, and
count as what they are clamped to, in every kind of grid: few shares, shares on
every SM (none left for the own rows), several waves, and the own rows in a
launch of their own (more than 1,024 requests)."""

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


# (8 requests of 32/8 heads behind 32,768 rows: 19 shares of 8 KV heads fill 152 SMs)
GRIDS = [(3, 8, 2, 64, 300), (8, 32, 8, 128, 32768), (40, 14, 2, 64, 20000), (1, 8, 8, 64, 9000), (70, 32, 8, 128, 4000),
         (1025, 4, 2, 64, 300)]


@pytest.mark.parametrize("Hq,Hkv,D,B,P", [(Hq, Hkv, D, B, P) for B, Hq, Hkv, D, P in GRIDS])
@pytest.mark.parametrize("kind", ["zero", "negative", "one negative", "long", "one long"])
def test_clamped_lengths_are_reported(Hq, Hkv, D, B, P, kind):
    S = 40
    lens = {"zero": [0] * B, "negative": [-1] * B, "one negative": [0] * (B - 1) + [-2 ** 31], "long": [S + 1] * B,
            "one long": [0] * (B - 1) + [2 ** 31 - 1]}[kind]
    q = inputs.randn((B, Hq, 1, D), 41, BF16, DEV)
    kp, vp = (inputs.randn((Hkv, P, D), s, BF16, DEV) for s in (42, 43))
    k, v = (inputs.randn((B, Hkv, S, D), s, BF16, DEV) for s in (44, 45))
    ws = binding.decode_shared_prefix_workspace(B, Hq, Hkv, D, P, S)
    ws[256:] = 0xFF
    o = binding.decode_shared_prefix(q, kp, vp, k, v, kv_lens=i32(lens), workspace=ws)
    assert binding.gqa_attn_read_device_status(ws) == (0 if kind == "zero" else binding.GQA_DEV_KVLEN_CLAMPED)
    some = sorted({0, B // 2, B - 1})
    ref = oracle.attention_shared_prefix(f64(q)[some], f64(kp), f64(vp), f64(k)[some], f64(v)[some],
                                         [min(max(lens[b], 0), S) for b in some], D ** -0.5)
    parity.check(f64(o)[some], ref, "bf16")
