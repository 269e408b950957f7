"""Attention of drafted rows (gqa_attn_decode_tree, _paged) on the GPU against the
64-bit oracle, under the bounds of a bf16 decode (tests/parity.py).  Rows past every
length are NaN, and so are keys of drafted rows that no query sees."""

import numpy as np
import pytest
import torch

import oracle
import parity
from gqa_attention_kv_decode_gb300 import binding, inputs

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16 = torch.bfloat16
SENTINEL = 3.0


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def f64(t):
    return t.detach().float().cpu().numpy()


def i32(a):
    return None if a is None else torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)


def tree_masks(rng, B, N, Tq, q_lens, tree_lens, density=None):
    """int32 [B, Tq, words]: ancestor masks of random trees, or (density) any bits.
    Bits past tree_lens and rows past q_lens are set at random."""
    words = -(-N // 32)
    mask = rng.integers(-2 ** 31, 2 ** 31, (B, Tq, words)).astype(np.int32)
    for b in range(B):
        n, q = int(tree_lens[b]), int(q_lens[b])
        parents = np.array([[-1] + [int(rng.integers(max(-1, i - 6), i)) for i in range(1, max(n, 1))]])
        rows, _, _ = oracle.tree_tables(parents, [n], [q], np.zeros((1, max(q, 1), -(-max(n, 1) // 32)), np.int32))
        for i in range(q):
            for c in range(n):
                on = rng.random() < density if density is not None else (int(rows[0, i, c // 32]) >> (c % 32)) & 1
                bit = np.int64(1) << (c % 32)
                word = np.int64(np.uint32(mask[b, i, c // 32]))
                mask[b, i, c // 32] = np.uint32((word | bit) if on else (word & ~bit)).astype(np.int32)
    return mask


class Case:
    def __init__(self, B, Hq, Hkv, D, Tq, kv_lens, q_lens=None, tree_lens=None, N=None, mask="tree", S=None, seed=0):
        rng = np.random.default_rng(seed + 17)
        self.B, self.Hkv, self.D = B, Hkv, D
        self.kv_lens = [int(x) for x in kv_lens]
        self.S = max(max(self.kv_lens), 1) if S is None else S
        ql = [Tq] * B if q_lens is None else [int(x) for x in q_lens]
        ql = [min(a, b) for a, b in zip(ql, self.kv_lens)]
        self.q_lens, self.tree_lens = q_lens, tree_lens
        nl = ql if tree_lens is None else [int(x) for x in tree_lens]
        N = max(max(nl), Tq, 1) if N is None else N
        self.mask = None
        if mask is not None:
            self.mask = tree_masks(rng, B, N, Tq, ql, nl, None if mask == "tree" else float(mask))
        self.q = inputs.randn((B, Hq, Tq, D), 700 + seed, BF16, DEV)
        self.k, self.v = (inputs.randn((B, Hkv, self.S, D), 700 + seed + i, BF16, DEV) for i in (1, 2))
        for b in range(B):  # queries past the lengths too
            self.q[b, :, ql[b]:] = float("nan")
        inputs.poison_tail(self.k, self.kv_lens)
        inputs.poison_tail(self.v, self.kv_lens)
        if self.mask is not None:
            for b in range(B):
                see = oracle.tree_visible(self.mask[b], Tq, ql[b], nl[b], self.kv_lens[b])
                for j in range(self.kv_lens[b] - nl[b], self.kv_lens[b]):
                    if ql[b] and not see[:, j].any():
                        self.k[b, :, j] = float("nan")
        self.scale = D ** -0.5
        self.o = torch.full_like(self.q, SENTINEL)

    def oracle(self):
        z = lambda t: np.nan_to_num(f64(t))  # noqa: E731  (NaN rows are never visible)
        return oracle.attention_tree(z(self.q), z(self.k), z(self.v), self.mask, self.q_lens, self.tree_lens,
                                     self.kv_lens, self.scale, np.full(self.q.shape, SENTINEL))

    def workspace(self, max_kv=None):
        B, Hq, Tq, D = self.q.shape
        return binding.decode_tree_workspace(B, Hq, self.Hkv, D, Tq, self.S if max_kv is None else max_kv)

    def args(self):
        return i32(self.mask), i32(self.q_lens), i32(self.tree_lens), i32(self.kv_lens)

    def dense(self, ws=None, max_kv=None, stream=None):
        ws = self.workspace(max_kv) if ws is None else ws
        o = self.o.clone()
        binding.gqa_attn_decode_tree(self.q, self.k, self.v, *self.args(), o, self.scale, ws, max_kv, stream)
        return o, binding.gqa_attn_read_device_status(ws, stream)

    def pools(self, bs, seed=1, spare=3):
        """The cache scattered over a pool; unused table entries point outside of it."""
        nb = -(-self.S // bs)
        n = self.B * nb + spare
        order = np.random.default_rng(seed).permutation(n)
        pools = [torch.full((n, self.Hkv, bs, self.D), float("nan"), dtype=BF16, device=DEV) for _ in range(2)]
        table, at = np.full((self.B, nb), -5), 0
        for b in range(self.B):
            for i in range(-(-self.kv_lens[b] // bs)):
                blk, m = int(order[at]), min(bs, self.S - i * bs)
                at += 1
                table[b, i] = blk
                for pool, x in zip(pools, (self.k, self.v)):
                    pool[blk, :, :m] = x[b, :, i * bs:i * bs + m]
        return *pools, i32(table)

    def paged(self, bs, ws=None, pools=None):
        kp, vp, table = self.pools(bs) if pools is None else pools
        ws = self.workspace(table.shape[1] * bs) if ws is None else ws
        o = self.o.clone()
        binding.gqa_attn_decode_tree_paged(self.q, kp, vp, table, *self.args(), o, self.scale, ws)
        return o, binding.gqa_attn_read_device_status(ws)

    def check(self, bs=None):
        """As planned, as one list over all SMs, and in clusters of two and of eight a unit."""
        ref, status = self.oracle()
        units = self.B * self.Hkv * -(-self.q.shape[1] // self.Hkv * self.q.shape[2] // 256)
        for split in (0, 1, 2, 8) if units <= 600 else (0, 1):
            with binding.plan_override(prefill_kv_split=split):
                o, seen = self.dense()
            parity.check(f64(o), ref, "bf16", f"dense, {split}")
            assert seen == status
        if bs is not None:
            o, seen = self.paged(bs)
            parity.check(f64(o), ref, "bf16", "paged")
            assert seen == status


def lens_of(B, lo, hi, seed=0):
    lens = np.random.default_rng(seed).integers(lo, hi + 1, B)
    lens[seed % B] = hi
    return lens


GEOMETRY = [(14, 2, 64), (28, 4, 128), (32, 8, 128), (8, 8, 64), (5, 5, 128), (24, 1, 64), (130, 1, 128), (33, 3, 64)]


@pytest.mark.parametrize("Hq,Hkv,D", GEOMETRY)
@pytest.mark.parametrize("B,Tq", [(1, 1), (1, 8), (3, 26), (2, 61)])
def test_geometries(Hq, Hkv, D, B, Tq):
    Case(B, Hq, Hkv, D, Tq, lens_of(B, Tq, 500, Tq), seed=B).check(64)


@pytest.mark.parametrize("L", [9, 10, 63, 64, 65, 127, 128, 129, 136, 137, 255, 256, 257, 384, 1000, 1023, 1025, 2049])
@pytest.mark.parametrize("Hq,Hkv,D,Tq", [(14, 2, 64, 9), (32, 8, 128, 9), (8, 2, 128, 40)])
def test_lengths_around_the_tiles(L, Hq, Hkv, D, Tq):
    Tq = min(Tq, L)
    Case(2, Hq, Hkv, D, Tq, [L, max(Tq, L - 3)], S=L + 70, seed=L).check(128)


@pytest.mark.parametrize("rows", [1, 2, 31, 32, 33, 63, 64, 65, 96, 127, 128, 129, 255, 256, 257, 384, 385, 512, 600])
@pytest.mark.parametrize("D", [64, 128])
def test_row_tiles(rows, D):
    """As many query rows of a KV head as fill tiles of 32, 128 and 256 rows, and one more or fewer."""
    Case(1, 2, 2, D, rows, [rows + 200], seed=rows).check()


@pytest.mark.parametrize("Hq,Hkv,D,Tq", [(4, 1, 64, 3), (4, 1, 128, 16), (8, 2, 64, 50), (4, 1, 128, 64), (6, 1, 128, 70),
                                         (16, 1, 64, 40)])
@pytest.mark.parametrize("lens", [[9000], [5000, 70, 1153, 0, 130], [1025, 1100], [33000]])
def test_few_long_units(Hq, Hkv, D, Tq, lens):
    """Many partials of a unit, joined by many warps; beside them units of one tile, of two and of none."""
    q_lens = [min(Tq, n) for n in lens]
    q_lens[-1] = min(q_lens[-1], max(1, Tq - 2))
    Case(len(lens), Hq, Hkv, D, Tq, lens, q_lens, seed=Tq).check(64)


@pytest.mark.parametrize("Hq,Hkv,D,Tq,lens", [(2, 1, 64, 1024, [1024, 1500]), (4, 2, 128, 700, [701, 2000]),
                                              (8, 1, 128, 333, [333, 900, 400]), (3, 1, 64, 1000, [5000])])
@pytest.mark.parametrize("kind", ["tree", None])
def test_large_trees(Hq, Hkv, D, Tq, lens, kind):
    """Masks over many key tiles, from every place in a tile, alone and behind other rows; chains as long."""
    Case(len(lens), Hq, Hkv, D, Tq, lens, mask=kind, seed=Tq).check(64)


@pytest.mark.parametrize("bs", [64, 128, 192, 448])
@pytest.mark.parametrize("D", [64, 128])
def test_block_sizes(bs, D):
    Case(3, 16, 4, D, 12, lens_of(3, 12, 900, bs), seed=bs).check(bs)


@pytest.mark.parametrize("Hq,Hkv,D", [(14, 2, 64), (32, 8, 128), (28, 4, 128)])
def test_ragged_queries(Hq, Hkv, D):
    """Requests with one query, some, all and none, without keys, and with nothing before the tree."""
    Case(8, Hq, Hkv, D, 20, [300, 77, 20, 1, 0, 40, 555, 19], [1, 7, 20, 1, 0, 0, 13, 19], seed=3).check(64)


@pytest.mark.parametrize("Hq,Hkv,D,Tq", [(14, 2, 64, 5), (32, 8, 128, 64), (28, 4, 128, 300)])
def test_chains(Hq, Hkv, D, Tq):
    """Without a mask every query sees the rows up to its own."""
    Case(3, Hq, Hkv, D, Tq, [Tq, Tq + 1, 700], mask=None).check(64)
    Case(3, Hq, Hkv, D, Tq, [Tq, Tq + 130, 700], [Tq, 1, Tq // 2], mask=None).check(64)


@pytest.mark.parametrize("N,Tq,tree,ql", [(40, 8, [40, 20, 8], [8, 8, 3]), (100, 10, [100, 64, 33], [10, 10, 1]),
                                          (200, 16, [200, 130, 16], [16, 16, 16])])
@pytest.mark.parametrize("D", [64, 128])
def test_queries_that_are_the_last_nodes_of_a_larger_tree(N, Tq, tree, ql, D):
    Case(3, 8, 2, D, Tq, [600, 131, 200], ql, tree, N).check(64)


@pytest.mark.parametrize("density", [0.0, 0.03, 0.5, 1.0])
@pytest.mark.parametrize("D", [64, 128])
def test_any_mask(density, D):
    """Masks of any bits; with nothing before the tree, rows that see nothing at all are zeros."""
    c = Case(4, 8, 2, D, 33, [33, 100, 161, 34], mask=str(density), seed=int(density * 100))
    c.check(64)


def test_status_of_an_empty_row_alone():
    c = Case(2, 8, 2, 64, 4, [4, 90], mask="1.0")
    c.mask[0, 2] = 0
    c.check(64)
    assert c.dense()[1] == binding.GQA_DEV_EMPTY_REQUEST


@pytest.mark.parametrize("D", [64, 128])
def test_peaked_scores(D):
    """Scores that grow along the keys raise the running maximum over and over; the
    largest are drafted rows that some queries do not see."""
    c = Case(2, 8, 2, D, 24, [1500, 1399], seed=9)
    c.k = (c.k.float() * torch.linspace(0.5, 4.0, c.S, device=DEV)[:, None]).to(BF16)
    c.check(64)


@pytest.mark.parametrize("fill", [30.0, -30.0])
def test_large_values(fill):
    """Sums and products in 32 bits: values far from one in every row of V and in one of K."""
    c = Case(2, 8, 2, 128, 6, [400, 128])
    c.v = (c.v.float() * 1e20).to(BF16)
    c.k[:, :, 5] = fill
    ref, _ = c.oracle()
    o, _ = c.dense()
    parity.check(f64(o) / 1e20, ref / 1e20, "bf16")


@pytest.mark.parametrize("B", [64, 300])
def test_many_short_requests(B):
    lens = lens_of(B, 3, 140, B)
    ql = np.minimum(np.random.default_rng(B).integers(0, 6, B), lens)
    Case(B, 8, 2, 64, 5, lens, ql, seed=B).check(64)
    Case(B, 8, 2, 128, 5, lens, ql, mask=None, seed=B).check(64)


def test_more_requests_than_threads():
    B = 2500
    lens = lens_of(B, 0, 70, 5)
    ql = np.minimum(np.random.default_rng(8).integers(0, 4, B), lens)
    Case(B, 4, 2, 64, 3, lens, ql, seed=5).check()


@pytest.mark.parametrize("D", [64, 128])
def test_long_caches_in_many_shares(D):
    c = Case(2, 8, 2, D, 16, [30011, 4097], seed=D)
    c.check(64)


def test_clamped_lengths():
    c = Case(3, 8, 2, 64, 6, [200, 90, 6], [6, 3, 6])
    c.kv_lens, c.q_lens = [5000, 90, 2], [6, -3, 6]  # (the rows past 200 are not there: nothing is poisoned)
    c.k, c.v, c.q = (torch.nan_to_num(x) for x in (c.k, c.v, c.q))
    ref, status = c.oracle()
    assert status == binding.GQA_DEV_KVLEN_CLAMPED
    o, seen = c.dense()
    parity.check(f64(o), ref, "bf16")
    assert seen == status


def test_a_shorter_bound_than_the_cache():
    c = Case(2, 8, 2, 128, 6, [200, 90], S=1000)
    o, seen = c.dense(max_kv=200)
    parity.check(f64(o), c.oracle()[0], "bf16")
    assert seen == 0


def test_bad_block_ids():
    c = Case(2, 8, 2, 64, 4, [200, 190])
    kp, vp, table = c.pools(64)
    table[1, 1] = 1 << 20
    o, seen = c.paged(64, pools=(kp, vp, table))
    assert seen == binding.GQA_DEV_BAD_BLOCK
    parity.check(f64(o)[:1], c.oracle()[0][:1], "bf16")


def test_offsets_past_32_bits():
    """Blocks behind the first 2^32 elements of a pool."""
    Hkv, D, bs, n = 8, 128, 64, 66_000
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 20 GB")
    c = Case(2, 16, Hkv, D, 7, [300, 130])
    kp, vp, table = c.pools(bs)
    far_k, far_v = (torch.zeros((n, Hkv, bs, D), dtype=BF16, device=DEV) for _ in range(2))
    m = kp.shape[0]
    far_k[n - m:], far_v[n - m:] = kp, vp
    o, _ = c.paged(bs, pools=(far_k, far_v, torch.where(table >= 0, table + (n - m), table)))
    parity.check(f64(o), c.oracle()[0], "bf16")


def test_the_same_bits_each_time():
    c = Case(5, 28, 4, 128, 20, lens_of(5, 20, 3000))
    ws = c.workspace()
    first = c.dense(ws)[0]
    for _ in range(4):
        assert torch.equal(c.dense(ws)[0], first)


def test_streams_graphs_and_growing_lengths():
    """A captured call replayed as lengths and masks change, beside another with a
    workspace of its own on another stream."""
    c, d = Case(4, 8, 2, 128, 8, [900, 200, 64, 8], seed=1), Case(3, 14, 2, 64, 30, [700, 31, 400], seed=2)
    caps = []
    for x, side in ((c, torch.cuda.Stream()), (d, torch.cuda.Stream())):
        ws, o, a = x.workspace(), x.o.clone(), x.args()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            binding.gqa_attn_decode_tree(x.q, x.k, x.v, *a, o, x.scale, ws)
        caps.append((x, graph, ws, o, a, side))
    for step in range(3):
        torch.cuda.synchronize()
        for x, graph, ws, o, a, side in caps:
            with torch.cuda.stream(side):
                for _ in range(5):
                    graph.replay()
        torch.cuda.synchronize()
        for x, graph, ws, o, a, side in caps:
            parity.check(f64(o), x.oracle()[0], "bf16", f"step {step}")
            x.kv_lens = [max(8, n - 7 * (step + 1)) if n > 40 else n for n in x.kv_lens]
            for t in (x.q, x.k):  # (in place: the captured calls read them; every drafted row may now be seen)
                t.copy_(torch.nan_to_num(t))
            a[3].copy_(i32(x.kv_lens))
            x.mask = np.roll(x.mask, 1, axis=1)
            a[0].copy_(i32(x.mask))
            o.fill_(SENTINEL)


def test_refusals():
    c = Case(2, 8, 2, 64, 4, [100, 50])
    m, ql, tl, kl = c.args()
    ws, o = c.workspace(), torch.full_like(c.q, SENTINEL)

    def refused(status, **kw):
        a = dict(q=c.q, k=c.k, v=c.v, m=m, ql=ql, tl=tl, kl=kl, o=o, ws=ws) | kw
        with pytest.raises(binding.GqaAttnError) as e:
            binding.gqa_attn_decode_tree(a["q"], a["k"], a["v"], a["m"], a["ql"], a["tl"], a["kl"], a["o"], c.scale, a["ws"])
        torch.cuda.synchronize()
        assert e.value.status == status
        assert (o == SENTINEL).all()

    refused(binding.GQA_ERR_INVALID_ARG, m=None, tl=kl)  # tree lengths without a mask
    refused(binding.GQA_ERR_INVALID_ARG, m=m.expand(2, 4, 1).repeat(1, 1, 33))
    refused(binding.GQA_ERR_NOT_DEVICE_PTR, q=c.q.cpu())
    refused(binding.GQA_ERR_NOT_DEVICE_PTR, m=m.cpu())
    refused(binding.GQA_ERR_NOT_DEVICE_PTR, kl=kl.cpu())
    refused(binding.GQA_ERR_WORKSPACE, ws=ws[:128])
    refused(binding.GQA_ERR_WORKSPACE, ws=ws[1:])
    refused(binding.GQA_ERR_UNSUPPORTED, q=c.q.float(), k=c.k.float(), v=c.v.float(), o=o.float())
    big = Case(1, 2, 2, 64, 40, [60])
    with pytest.raises(binding.GqaAttnError) as e:  # 32 bits for 40 queries' own rows
        binding.decode_tree(big.q, big.k, big.v, i32([60]), i32(np.zeros((1, 40, 1))))
    assert e.value.status == binding.GQA_ERR_INVALID_ARG
    kp, vp, table = c.pools(64)
    with pytest.raises(binding.GqaAttnError) as e:
        binding.decode_tree_paged(c.q, kp[:, :, :32].contiguous(), vp[:, :, :32].contiguous(), table, kl, m)
    assert e.value.status == binding.GQA_ERR_UNSUPPORTED


def test_convenience_calls():
    c = Case(2, 8, 2, 64, 4, [100, 50])
    m, ql, tl, kl = c.args()
    ref = c.oracle()[0]
    parity.check(f64(binding.decode_tree(c.q, c.k, c.v, kl, m)), ref, "bf16")
    kp, vp, table = c.pools(64)
    parity.check(f64(binding.decode_tree_paged(c.q, kp, vp, table, kl, m)), ref, "bf16")
