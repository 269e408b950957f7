"""Steps that verify drafted tokens, in one captured graph: tables of the step and of
the trees, new rows into a paged cache, attention of the trees, accepted rows moved
together, requests that fork, end or give drafted rows' blocks back, and the copies
of pages that this needs.  Beside it a plain model of every request's rows."""

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


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)


def ints(t):
    return t.cpu().numpy()


def f64(t):
    return t.detach().float().cpu().numpy()


class Server:
    """B request slots, trees of up to N nodes, two layers' caches of blocks of `bs` rows."""

    def __init__(self, B, Hq, Hkv, D, N, bs, mb, pool):
        self.B, self.Hq, self.Hkv, self.D, self.N, self.bs = B, Hq, Hkv, D, N, bs
        self.T = B * N
        z = lambda *s: torch.zeros(s, dtype=torch.int32, device=DEV)  # noqa: E731
        self.lens, self.new, self.table = z(B), z(B), z(B, mb)
        self.stack, self.count, self.shared = i32(np.random.default_rng(0).permutation(pool)), i32([pool]), z(pool)
        self.kv, self.q_lens, self.starts = z(B), z(B), z(B + 1)
        self.pos, self.slots, self.q_slots = z(self.T), z(self.T), z(self.T)
        self.parents, self.mask = z(B, N), z(B, N, -(-N // 32))
        self.path, self.keep, self.kept = z(B, N), z(B), z(B)
        self.src, self.table2, self.lens2 = z(B), z(B, mb), z(B)
        self.csrc, self.cdst, self.crows = z(B), z(B), z(B)
        self.x = [torch.zeros((self.T, (Hq + 2 * Hkv) * D), dtype=BF16, device=DEV) for _ in range(2)]
        self.k, self.v = (torch.full((2, pool, Hkv, bs, D), float("nan"), dtype=BF16, device=DEV) for _ in range(2))
        self.q = [torch.zeros((B, Hq, N, D), dtype=BF16, device=DEV) for _ in range(2)]
        self.o = [torch.zeros((B, Hq, N, D), dtype=BF16, device=DEV) for _ in range(2)]
        self.cs = binding.rope_table(mb * bs, D)
        self.max_kv = mb * bs
        self.ws = binding.decode_tree_workspace(B, Hq, Hkv, D, N, self.max_kv)

    def heads(self, layer):
        Hq, Hkv, D = self.Hq, self.Hkv, self.D
        return (t.unflatten(1, (-1, D)) for t in self.x[layer].split([Hq * D, Hkv * D, Hkv * D], dim=1))

    def step(self):
        b = binding
        b.gqa_attn_step_tables(self.lens, self.new, self.table, self.stack, self.count, self.kv, self.q_lens, self.starts,
                               self.pos, self.slots, self.q_slots, self.count, self.bs, self.N, self.ws)
        b.gqa_attn_tree_tables(self.parents, self.q_lens, None, self.kv, self.starts, self.mask, self.pos, self.ws)
        for layer in range(2):
            q, k, v = self.heads(layer)
            b.gqa_attn_rope_append(q, k, v, None, None, 0.0, self.cs, self.pos, self.slots, self.q_slots, self.q[layer],
                                   self.k[layer], self.v[layer], False, self.ws)
            b.gqa_attn_decode_tree_paged(self.q[layer], self.k[layer], self.v[layer], self.table, self.mask, self.q_lens,
                                         None, self.kv, self.o[layer], self.D ** -0.5, self.ws, self.max_kv)
        b.gqa_attn_compact_rows(self.path, self.keep, self.q_lens, self.kv, self.table, self.k, self.v, self.kept, self.ws)
        # (a fork keeps all that its source keeps; `kept` is by source, keep_lens by new request)
        keep = torch.gather(self.kept, 0, self.src.clamp(min=0).long())
        b.gqa_attn_fork_tables(self.src, keep, self.kv, self.table, self.shared, self.stack, self.count, self.table2,
                               self.lens2, self.shared, self.stack, self.count, self.csrc, self.cdst, self.crows, self.bs,
                               self.ws)
        b.gqa_attn_copy_blocks(self.csrc, self.cdst, self.crows, self.k, self.v, self.ws)
        self.table.copy_(self.table2)
        self.lens.copy_(self.lens2)


@pytest.mark.parametrize("B,Hq,Hkv,D,N,bs,mb", [(6, 14, 2, 64, 9, 64, 4), (4, 8, 2, 128, 40, 64, 6)])
def test_steps(B, Hq, Hkv, D, N, bs, mb):
    s = Server(B, Hq, Hkv, D, N, bs, mb, B * mb + 8)
    rng = np.random.default_rng(B)
    pool = s.stack.numel()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        s.step()
    rows = [[[np.zeros((0, Hkv, D))] * 2 for _ in range(2)] for _ in range(B)]  # [request][layer][K, V]: [rows, Hkv, D]
    cs = f64(s.cs)
    for step in range(14):
        lens = np.array([len(r[0][0]) for r in rows])
        # prompts of a chain, then trees; a request near its end drafts nothing
        new = np.minimum(rng.integers(0 if step > 2 else 1, N + 1, B), mb * bs - lens)
        parents = np.stack([np.array([-1] + [int(rng.integers(max(0, i - 5), i)) for i in range(1, N)]) for _ in range(B)])
        if step == 0:
            parents = np.tile(np.arange(-1, N - 1), (B, 1))
        path, keep = np.full((B, N), -1), np.zeros(B, int)
        for b in range(B):  # a random way down the tree
            at, way = -1, []
            while True:
                below = [c for c in range(int(new[b])) if parents[b, c] == at]
                if not below or len(way) > 6 + 99 * (step == 0):
                    break
                at = int(rng.choice(below))
                way.append(at)
            path[b, :len(way)], keep[b] = way, len(way)
        src = np.where(rng.random(B) < 0.25, rng.integers(-1, B, B), np.arange(B))
        for t, a in ((s.new, new), (s.parents, parents), (s.path, path), (s.keep, keep), (s.src, src)):
            t.copy_(i32(a))
        for layer in range(2):
            s.x[layer].copy_(inputs.randn(s.x[layer].shape, 50 * step + layer, BF16, DEV))
            s.o[layer].fill_(3.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert binding.gqa_attn_read_device_status(s.ws) == 0
        assert (ints(s.q_lens) == new).all()
        starts = np.concatenate([[0], np.cumsum(new)])
        live = [slice(starts[b], starts[b + 1]) for b in range(B)]
        for b in range(B):
            depth = []
            for c in range(int(new[b])):
                depth.append(depth[parents[b, c]] + 1 if parents[b, c] >= 0 else 0)
            assert (ints(s.pos)[live[b]] == lens[b] + np.array(depth, int)).all()
        for layer in range(2):
            q, k, v = (f64(t) for t in s.heads(layer))
            pos = ints(s.pos)
            half = D // 2
            q, k = (oracle.rotate(t, cs[pos, :half], cs[pos, half:], False) for t in (q, k))
            k = f64(torch.from_numpy(k).to(BF16))
            for b in range(B):
                n, L = int(new[b]), int(lens[b] + new[b])
                if n == 0:
                    continue
                kk, vv = (np.concatenate([rows[b][layer][i], x[live[b]]]).transpose(1, 0, 2)[None]
                          for i, x in enumerate((k, v)))
                qq = f64(s.q[layer])[b:b + 1]
                want_q = q[live[b]].transpose(1, 0, 2)
                assert (np.abs(qq[0, :, :n] - want_q) <= 2.0 ** -8 * (1 + np.abs(want_q))).all()
                mask, _, _ = oracle.tree_tables(parents[b:b + 1], [n], None, np.zeros((1, N, s.mask.shape[2]), np.int32))
                ref, _ = oracle.attention_tree(qq, kk, vv, mask, [n], None, [L], D ** -0.5, np.full(qq.shape, 3.0))
                parity.check(f64(s.o[layer])[b:b + 1], ref, "bf16", f"step {step}, request {b}")
                rows[b][layer] = [np.concatenate([rows[b][layer][i], x[live[b]][path[b, :keep[b]]]]) for i, x in enumerate((k, v))]
        rows = [[list(x) for x in rows[a]] if a >= 0 else [[np.zeros((0, Hkv, D))] * 2 for _ in range(2)] for a in src]
        # the caches hold these rows, and the pool's blocks are all accounted for
        table, stack, count, shared = ints(s.table), ints(s.stack), int(s.count), ints(s.shared)
        held = np.zeros(pool, int)
        for b in range(B):
            n = len(rows[b][0][0])
            assert int(s.lens[b]) == n
            ids = table[b, :-(-n // bs)]
            held[ids] += 1
            for layer in range(2):
                for i, c in enumerate((s.k, s.v)):
                    got = f64(c[layer][i32(ids).long()].transpose(1, 2).reshape(-1, Hkv, D)[:n])
                    # (two roundings to bf16, of 32 and of 64 bits: a step of 2^-7 at most between them)
                    assert (np.abs(got - rows[b][layer][i]) <= 2.0 ** -7 * (1 + np.abs(got))).all()
                    rows[b][layer][i] = got
        assert len(set(stack[:count])) == count and not held[stack[:count]].any()
        assert ((held > 0).sum() + count == pool) and (shared == np.maximum(held - 1, 0)).all()


def test_beams_over_one_prompt():
    """One prompt, forked into eight, each of which goes on by itself; half of them end."""
    Hq, Hkv, D, bs, mb, pool, P = 8, 2, 64, 64, 8, 40, 200
    r = np.random.default_rng(0)
    k, v = (inputs.randn((pool, Hkv, bs, D), s, BF16, DEV) for s in (1, 2))
    stack = r.permutation(pool)
    table = np.zeros((1, mb), int)
    table[0, :4] = stack[-4:]
    z = lambda *s: torch.zeros(s, dtype=torch.int32, device=DEV)  # noqa: E731
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    g_stack, count, shared = i32(stack), i32([pool - 4]), z(pool)
    t8, l8, cs, cd, cr = z(8, mb), z(8), z(8), z(8), z(8)
    binding.gqa_attn_fork_tables(i32([0] * 8), None, i32([P]), i32(table), shared, g_stack, count, t8, l8, shared, g_stack,
                                 count, cs, cd, cr, bs, ws)
    binding.gqa_attn_copy_blocks(cs, cd, cr, k, v, ws)
    assert ints(l8).tolist() == [P] * 8 and int(count) == pool - 4 - 7 and int(shared.sum()) == 3 * 7
    # one step of a token each
    q_lens, starts, pos, slots = z(8), z(9), z(8), z(8)
    binding.gqa_attn_step_tables(l8, i32([1] * 8), t8, g_stack, count, l8, q_lens, starts, pos, slots, None, count, bs, 1, ws)
    kn, vn = (inputs.randn((8, Hkv, D), s, BF16, DEV) for s in (3, 4))
    qn = inputs.randn((8, Hq, D), 5, BF16, DEV)
    q = torch.zeros((8, Hq, 1, D), dtype=BF16, device=DEV)
    binding.gqa_attn_rope_append(qn, kn, vn, None, None, 0.0, None, None, slots, None, q, k, v, False, ws)
    o = binding.decode_tree_paged(q, k, v, t8, l8)
    kk, vv = (f64(x[t8.long()].transpose(1, 2).reshape(8, Hkv, mb * bs, D)) for x in (k, v))
    assert (kk[:, :, P] == f64(kn)).all() and (kk[1:, :, :P] == kk[:1, :, :P]).all()
    ref, _ = oracle.attention_tree(f64(q), kk, vv, None, None, None, [P + 1] * 8, D ** -0.5, np.zeros(q.shape))
    parity.check(f64(o), ref, "bf16")
    # the decode of one query is the same attention
    parity.check(f64(binding.decode_paged(q, k, v, t8, l8, mb * bs)), ref, "bf16")
    t4, l4 = z(4, mb), z(4)
    binding.gqa_attn_fork_tables(i32([1, 3, 5, 7]), None, l8, t8, shared, g_stack, count, t4, l4, shared, g_stack, count,
                                 cs[:4], cd[:4], cr[:4], bs, ws)
    assert int(count) == pool - 4 - 7 + 4 and int(shared.sum()) == 3 * 3 and ints(cs)[:4].tolist() == [-1] * 4
    assert binding.gqa_attn_read_device_status(ws) == 0
