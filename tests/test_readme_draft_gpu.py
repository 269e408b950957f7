"""The draft step that the README prints, run as it is printed, against the plain
model of every request's rows."""

import os
import re

import pytest

import test_draft_step_gpu as draft
from gqa_attention_kv_decode_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def printed_parts():
    """Before the appends, for each layer, for all layers."""
    text = open(os.path.join(os.path.dirname(os.path.dirname(__file__)), "README.md")).read()
    blocks = [b for b in re.findall(r"^  ```\n(.*?)^  ```$", text, re.S | re.M) if "gqa_attn_tree_tables" in b]
    assert len(blocks) == 1
    parts = re.split(r"^#.*\n", "".join(line[2:] for line in blocks[0].splitlines(True)), flags=re.M)
    assert len(parts) == 3
    return parts


def printed_step(s):
    first, layer_part, last = printed_parts()
    names = {n: getattr(binding, n) for n in binding.EXPORTED if hasattr(binding, n)}
    names |= dict(parents=s.parents, q_lens=s.q_lens, lens=s.kv, q_starts=s.starts, tree_mask=s.mask, positions=s.pos,
                  ws=s.ws, table=s.table, scale=s.D ** -0.5, max_kv_len=s.max_kv, path=s.path, n_keep=s.keep,
                  k_pools=s.k, v_pools=s.v, kept_lens=s.kept, src=s.src, shared=s.shared, free_blocks=s.stack,
                  free_count=s.count, new_table=s.table2, new_lens=s.lens2, copy_src=s.csrc, copy_dst=s.cdst,
                  copy_rows=s.crows, block_size=s.bs)
    binding.gqa_attn_step_tables(s.lens, s.new, s.table, s.stack, s.count, s.kv, s.q_lens, s.starts, s.pos, s.slots,
                                 s.q_slots, s.count, s.bs, s.N, s.ws)
    exec(first, names)
    for layer in range(2):
        q, k, v = s.heads(layer)
        binding.gqa_attn_rope_append(q, k, v, None, None, 0.0, s.cs, s.pos, s.slots, s.q_slots, s.q[layer], s.k[layer],
                                     s.v[layer], False, s.ws)
        names |= dict(q_out=s.q[layer], k_pool=s.k[layer], v_pool=s.v[layer], o=s.o[layer])
        exec(layer_part, names)
    exec(last, names)
    s.table.copy_(s.table2)
    s.lens.copy_(s.lens2)


def test_the_printed_draft_step(monkeypatch):
    monkeypatch.setattr(draft.Server, "step", printed_step)
    draft.test_steps(5, 8, 2, 64, 20, 64, 4)
