"""The decode step that the README prints, run as it is printed: every request's
own keys rotated at their positions behind the shared prefix, and attended."""

import os
import re

import numpy as np
import pytest
import torch

import oracle
import parity
from gqa_attention_kv_decode_gb300 import binding
from test_serving_step_gpu import BF16, DEV, Model, f64, i32, ints, ulp_close

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def printed_step():
    text = open(os.path.join(os.path.dirname(os.path.dirname(__file__)), "README.md")).read()
    blocks = [b for b in re.findall(r"^  ```\n(.*?)^  ```$", text, re.S | re.M) if "gqa_attn_step_tables" in b]
    assert len(blocks) == 1
    return "\n".join(line[2:] for line in blocks[0].splitlines())


@pytest.mark.parametrize("offset", ["added", "in the angle table"])
def test_the_printed_step(offset):
    Hq, Hkv, D, B, bs, P, mb = 32, 8, 128, 5, 64, 150, 2
    m = Model(Hq, Hkv, D, False, 1000, 11)
    npb = -(-P // bs)
    pool = npb + B * mb
    kp, vp = (torch.randn((pool, Hkv, bs, D), generator=torch.Generator().manual_seed(s)).to(BF16).to(DEV)
              for s in (1, 2))
    order = np.random.default_rng(2).permutation(pool)
    names = {n: getattr(binding, n) for n in binding.EXPORTED if hasattr(binding, n)}
    names |= dict(lens=i32([0] * B), new_lens=i32([1] * B), table=torch.zeros((B, mb), dtype=torch.int32, device=DEV),
                  free_blocks=i32(np.concatenate([order[npb:], order[:npb]])), free_count=i32([pool - npb]),
                  q_lens=ints(B), q_starts=ints(B + 1), positions=ints(B), slots=ints(B), q_slots=ints(B),
                  block_size=bs, q_norm=m.wq, k_norm=m.wk, eps=m.eps, cos_sin=m.cs, k_pool=kp, v_pool=vp,
                  q_out=torch.zeros((B, Hq, 1, D), dtype=BF16, device=DEV),
                  o=torch.zeros((B, Hq, 1, D), dtype=BF16, device=DEV), prefix_table=i32(order[:npb]),
                  prefix_len=i32([P]), scale=D ** -0.5, max_prefix_len=npb * bs, max_kv_len=mb * bs,
                  ws=binding.decode_shared_prefix_workspace(B, Hq, Hkv, D, npb * bs, mb * bs))
    code = printed_step()
    if offset != "added":  # the README's other form
        code, n = re.subn(r"^behind = .*$", "behind, cos_sin = positions, all_angles[P:]", code, flags=re.M)
        assert n == 1
        names |= dict(all_angles=m.cs, P=P)
    hist = [([], []) for _ in range(B)]
    for n in range(70):
        x = m.project(B, n)
        names["q"], names["k"], names["v"] = m.views(x)
        exec(code, names)
        kk, vv = m.keys(x, np.full(B, P + n))
        for b in range(B):
            hist[b][0].append(kk[b])
            hist[b][1].append(vv[b])
    torch.cuda.synchronize()
    table, ptable = names["table"].long(), names["prefix_table"].long()
    own = [f64(t[table].transpose(1, 2).reshape(B, Hkv, mb * bs, D)[:, :, :70]) for t in (kp, vp)]
    shared = [f64(t[ptable].transpose(0, 1).reshape(Hkv, npb * bs, D)[:, :P]) for t in (kp, vp)]
    for b in range(B):
        assert ulp_close(own[0][b], np.stack(hist[b][0], 1)) and (own[1][b] == np.stack(hist[b][1], 1)).all()
    q, _, _ = m.views(x)
    cs = f64(m.cs)[np.full(B, P + 69)]
    want = oracle.rotate(oracle.rms_norm(f64(q), f64(m.wq), m.eps), cs[:, :D // 2], cs[:, D // 2:], False)
    assert ulp_close(f64(names["q_out"])[:, :, 0], want)
    ref = oracle.attention_shared_prefix(f64(names["q_out"]), *shared, *own, [70] * B, D ** -0.5)
    parity.check(f64(names["o"]), ref, "bf16")
    assert binding.gqa_attn_read_device_status(names["ws"]) == 0
