"""Tree tables, accepted rows, forked tables and copied pages on the GPU: equal to
the oracle, bit by bit, and nothing else changed."""

import numpy as np
import pytest
import torch

import oracle
from gqa_attention_kv_decode_gb300 import binding, inputs

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def i32(a):
    return None if a is None else torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)


def ints(t):
    return t.cpu().numpy()


@pytest.fixture
def ws():
    return torch.zeros(256, dtype=torch.uint8, device=DEV)


def status(ws):
    return binding.gqa_attn_read_device_status(ws)


# ---------------------------------------------------------------- tree tables

def run_tables(ws, parents, tree_lens, q_lens, Tq, kv_lens=None, q_starts=None, T=0, seed=0):
    B, N = np.asarray(parents).shape
    r = np.random.default_rng(seed)
    mask = r.integers(-9, 9, (B, Tq, -(-N // 32))).astype(np.int32)
    pos = None if kv_lens is None else r.integers(-9, 9, T).astype(np.int32)
    gm, gp = i32(mask), i32(pos)
    binding.gqa_attn_tree_tables(i32(parents), i32(tree_lens), i32(q_lens), i32(kv_lens), i32(q_starts), gm, gp, ws)
    want_mask, want_pos, want = oracle.tree_tables(parents, tree_lens, q_lens, mask, kv_lens, q_starts, pos)
    assert (ints(gm) == want_mask).all()
    if pos is not None:
        assert (ints(gp) == want_pos).all()
    assert status(ws) == want
    return want


def random_parents(r, B, N, back):
    lo = np.maximum(np.arange(N) - back, -1)
    p = np.floor(lo + r.random((B, N)) * (np.arange(N) - lo)).astype(int)
    p[:, 0] = -1
    return p


@pytest.mark.parametrize("N", [1, 2, 26, 31, 32, 33, 63, 64, 65, 100, 256, 257, 1000, 1024])
@pytest.mark.parametrize("back", [1, 5, 2000])
def test_tree_tables(ws, N, back):
    """Chains, trees like drafts and random ones; every word border."""
    r = np.random.default_rng(N)
    B = 3
    n = np.array([N, max(N - 3, 0), N // 2])
    kv = n + r.integers(0, 500, B)
    run_tables(ws, random_parents(r, B, N, back), n, None, N, kv, [0, n[0], n[0] + n[1], n.sum()], int(n.sum()) + 2)


@pytest.mark.parametrize("B,N,Tq", [(1, 64, 5), (40, 50, 10), (300, 26, 26), (700, 70, 1)])
def test_tree_tables_of_a_batch(ws, B, N, Tq):
    r = np.random.default_rng(B)
    n = r.integers(0, N + 1, B)
    q = np.minimum(r.integers(0, Tq + 1, B), n)
    starts = np.concatenate([[0], np.cumsum(q)])
    assert run_tables(ws, random_parents(r, B, N, 7), n, q, Tq, n + r.integers(0, 9000, B), starts, int(starts[-1]) + 3) == 0


def test_tree_tables_bad_input(ws):
    C, X = binding.GQA_DEV_KVLEN_CLAMPED, binding.GQA_DEV_BAD_INDEX
    good = random_parents(np.random.default_rng(0), 2, 40, 5)
    bad = good.copy()
    bad[0, 7], bad[0, 35], bad[1, 3], bad[1, 39] = 7, 36, -2, 1 << 30
    assert run_tables(ws, bad, [40, 40], None, 40) == X
    binding.gqa_attn_clear_device_status(ws)
    # (parents of nodes that are not there are not looked at)
    assert run_tables(ws, bad, [7, 3], None, 40) == 0
    for n, q in (([41, 2], [3, 2]), ([-1, 2], [0, 2]), ([40, 2], [3, 3]), ([40, 2], [-3, 1]), ([40, 40], [40, 13])):
        binding.gqa_attn_clear_device_status(ws)
        assert run_tables(ws, good, n, q, 12, [50, 60], [0, 12, 24], 24) == C
    binding.gqa_attn_clear_device_status(ws)
    assert run_tables(ws, good, [10, 9], None, 12, [9, 9], [0, 10, 19], 19) == C  # a tree longer than its request
    binding.gqa_attn_clear_device_status(ws)
    assert run_tables(ws, good, [10, 9], None, 12, [90, 90], [-3, 15, 19], 18) == 0  # positions past either end are left out


# ---------------------------------------------------------------- accepted rows

def bits(t):
    return t.contiguous().view(torch.int32 if t.dtype == torch.float32 else torch.int16).cpu().numpy()


def run_compact(ws, path, keep, tree_lens, kv_lens, table, k, v):
    want_k, want_v, want_lens, want = oracle.compact_rows(path, keep, tree_lens, kv_lens, table,
                                                          *(bits(x if x.dim() == 5 else x[None]) for x in (k, v)))
    out = i32(np.full(len(keep), -7))
    binding.gqa_attn_compact_rows(i32(path), i32(keep), i32(tree_lens), i32(kv_lens), i32(table), k, v, out, ws)
    assert (ints(out) == want_lens).all()
    assert (bits(k).reshape(want_k.shape) == want_k).all() and (bits(v).reshape(want_v.shape) == want_v).all()
    assert status(ws) == want
    return want


def random_paths(r, B, N, P):
    path = np.full((B, P), -1)
    keep = r.integers(0, min(N, P) + 1, B)
    for b in range(B):
        path[b, :keep[b]] = np.sort(r.choice(N, keep[b], replace=False))
    return path, keep


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,N,P,bs,layers,Hkv", [(1, 16, 5, 64, 28, 4), (5, 64, 20, 16, 3, 2), (40, 30, 30, 7, 2, 1),
                                                 (3, 200, 200, 64, 1, 8), (2, 1, 1, 1, 2, 5)])
def test_compact_paged(ws, dtype, D, B, N, P, bs, layers, Hkv):
    r = np.random.default_rng(B * N)
    path, keep = random_paths(r, B, N, P)
    lens = N + r.integers(0, 2 * bs + 1, B)
    mb = -(-int(lens.max()) // bs)
    pool = B * mb + 2
    table = r.permutation(pool)[:B * mb].reshape(B, mb)
    k, v = (inputs.randn((layers, pool, Hkv, bs, D), s, dtype, DEV) for s in (1, 2))
    assert run_compact(ws, path, keep, [N] * B, lens, table, k, v) == 0


@pytest.mark.parametrize("layers", [None, 3])
def test_compact_dense(ws, layers):
    r = np.random.default_rng(3)
    path, keep = random_paths(r, 6, 40, 12)
    shape = (6, 2, 111, 64) if layers is None else (layers, 6, 2, 111, 64)
    k, v = (inputs.randn(shape, s, torch.bfloat16, DEV) for s in (1, 2))
    assert run_compact(ws, path, keep, [40] * 6, r.integers(40, 112, 6), None, k, v) == 0


def test_compact_a_whole_tree_shifted_by_one(ws):
    """Every row but the first is both a source and a destination."""
    k, v = (inputs.randn((1, 300, 1, 64), s, torch.bfloat16, DEV)[:, :, :, None].expand(1, 300, 1, 64, 64).reshape(
        1, 1, 300 * 64, 64) for s in (1, 2))
    path = np.arange(1, 1001)[None]
    assert run_compact(ws, path, [1000], [1001], [5000], None, k, v) == 0


def test_compact_bad_input(ws):
    C, X, Bk = binding.GQA_DEV_KVLEN_CLAMPED, binding.GQA_DEV_BAD_INDEX, binding.GQA_DEV_BAD_BLOCK
    r = np.random.default_rng(5)
    table = r.permutation(9).reshape(3, 3)
    k, v = (inputs.randn((2, 9, 2, 16, 64), s, torch.bfloat16, DEV) for s in (1, 2))

    def run(path=((1, 2, 5), (0, 2, 9), (3, 4, 5)), keep=(3, 3, 3), tree=(10, 10, 10), lens=(40, 30, 20), t=table):
        binding.gqa_attn_clear_device_status(ws)
        return run_compact(ws, path, keep, tree, lens, t, k, v)

    assert run() == 0
    for p in ((2, 2, 5), (5, 2, 9), (1, 2, 10), (-1, 2, 3), (1, 2, 1 << 30)):
        assert run(path=((1, 2, 5), p, (3, 4, 5))) == X
    assert run(keep=(4, 3, 3)) == C and run(keep=(3, -1, 3)) == C and run(tree=(2, 10, 10), path=((0, 1, 5),) * 3) == C
    assert run(tree=(41, 10, 10)) == C and run(lens=(49, 30, 20)) == C and run(lens=(-1, 30, 20)) == C
    bad = table.copy()
    bad[1, 1] = 9  # rows 16 to 31
    assert run(t=bad) == Bk
    bad[1, 1] = -1
    assert run(t=bad, keep=(3, 2, 3)) == Bk


# ---------------------------------------------------------------- forks

def pool_of_requests(r, B_in, bs, mb, spare, families=True):
    """Old requests of families with shared first blocks: held_lens, table, shared, stack, count."""
    held = r.integers(0, mb * bs + 1, B_in)
    family = np.sort(r.integers(0, max(1, B_in // 3), B_in)) if families else np.arange(B_in)
    common = (r.integers(0, mb * bs + 1, B_in) // bs)[family] if families else np.zeros(B_in, int)
    n = 2 * B_in * mb + spare
    order = r.permutation(n)
    table, holders = np.full((B_in, mb), -3), np.zeros(n, int)
    for b in range(B_in):
        for j in range(-(-int(held[b]) // bs)):
            whole = j < common[b] and (j + 1) * bs <= held[b]
            table[b, j] = order[family[b] * mb + j] if whole else order[B_in * mb + b * mb + j]
            holders[table[b, j]] += 1
    stack = np.zeros(n, int)
    stack[:spare] = order[n - spare:]
    return held, table, np.maximum(holders - 1, 0), stack, spare


def run_fork(ws, src, keep, held, table, shared, stack, count, bs, in_place=False):
    B, mb = len(src), np.asarray(table).shape[1]
    before = np.random.default_rng(1).integers(-9, 9, (B, mb))
    want = oracle.fork_tables(src, keep, held, table, shared, stack, count, before, bs)
    g = {"shared": i32(shared), "free_blocks": i32(stack), "free_count": i32([count])}
    out = {"block_table": i32(before), "kv_lens": i32([-7] * B), "copy_src": i32([-7] * B), "copy_dst": i32([-7] * B),
           "copy_rows": i32([-7] * B)} | (g if in_place else {k: torch.full_like(v, -7) for k, v in g.items()})
    inputs_before = {k: v.clone() for k, v in g.items()}
    binding.gqa_attn_fork_tables(i32(src), i32(keep), i32(held), i32(table), g["shared"], g["free_blocks"], g["free_count"],
                                 out["block_table"], out["kv_lens"], out["shared"], out["free_blocks"], out["free_count"],
                                 out["copy_src"], out["copy_dst"], out["copy_rows"], bs, ws)
    for name, t in out.items():
        assert (ints(t) == want[name]).all(), name
    if not in_place:
        for k, v in inputs_before.items():
            assert torch.equal(g[k], v)
    assert status(ws) == want["status"]
    return want


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B_in,B,bs,mb", [(1, 1, 16, 3), (1, 9, 64, 5), (8, 8, 16, 40), (33, 20, 1, 12), (100, 150, 4, 33),
                                          (257, 300, 16, 6), (1100, 1030, 2, 3), (3, 2000, 8, 70), (2, 3, 1, 4100), (16, 15, 2, 384),
                                          (17, 16, 1, 130), (40, 5, 1, 900), (1, 1, 2, 129), (128, 100, 3, 200), (8192, 8192, 1, 2)])
def test_forks(ws, B_in, B, bs, mb, in_place):
    r = np.random.default_rng(B_in + B)
    held, table, shared, stack, count = pool_of_requests(r, B_in, bs, mb, B + 5)
    src = r.integers(-1, B_in, B)
    keep = np.floor(held[np.maximum(src, 0)] * np.where(r.random(B) < 0.5, 1.0, r.random(B))).astype(int)
    assert run_fork(ws, src, np.where(src < 0, 0, keep), held, table, shared, stack, count, bs, in_place)["status"] == 0


def test_everything_stays(ws):
    """Each request its own successor: no block moves, whatever is shared."""
    r = np.random.default_rng(2)
    held, table, shared, stack, count = pool_of_requests(r, 20, 8, 9, 4)
    w = run_fork(ws, np.arange(20), None, held, table, shared, stack, count, 8)
    assert (w["shared"] == shared).all() and w["free_count"][0] == count and (w["copy_src"] == -1).all()


def test_everything_ends(ws):
    """Every holder of every block gives it back: all of them are on the stack once."""
    r = np.random.default_rng(3)
    held, table, shared, stack, count = pool_of_requests(r, 30, 4, 11, 6)
    w = run_fork(ws, [-1] * 3, None, held, table, shared, stack, count, 4)
    n = int(w["free_count"][0])
    assert not w["shared"].any() and len(set(w["free_blocks"][:n])) == n
    assert set(w["free_blocks"][6:n]) == {int(x) for x in table[table >= 0]}


def test_blocks_shared_by_old_requests_and_cut(ws):
    """Requests that share a whole block and are all cut inside of it copy it each, and it is free afterwards."""
    table = [[0, 1], [0, 2], [0, 3]]
    w = run_fork(ws, [0, 1, 2, 0], [3, 2, 1, 3], [8, 8, 8], table, [2, 0, 0, 0, 0, 0, 0, 0], [4, 5, 6, 7, 0, 0, 0, 0], 4, 4)
    assert w["status"] == 0 and (w["copy_src"] == 0).all() and w["copy_dst"].tolist() == [7, 6, 5, 4]
    assert w["free_blocks"][:4].tolist() == [0, 1, 2, 3]


@pytest.mark.parametrize("in_place", [False, True])
def test_too_few_free_blocks(ws, in_place):
    r = np.random.default_rng(6)
    held, table, shared, stack, count = pool_of_requests(r, 12, 16, 5, 3)
    w = run_fork(ws, r.integers(0, 12, 40), None, held, table, shared, stack, count, 16, in_place)
    assert w["status"] == binding.GQA_DEV_OUT_OF_BLOCKS and (w["copy_src"] >= 0).sum() == 3


def test_fork_bad_input(ws):
    C, X, Bk = binding.GQA_DEV_KVLEN_CLAMPED, binding.GQA_DEV_BAD_INDEX, binding.GQA_DEV_BAD_BLOCK

    def run(src=(0, 1, 1), keep=(9, 7, 5), held=(10, 7), table=((0, 1, 2), (3, 4, -9)), shared=(0,) * 10,
            stack=(9, 8, 7, 6, 5, 0, 0, 0, 0, 0), count=5):
        binding.gqa_attn_clear_device_status(ws)
        return run_fork(ws, src, keep, held, table, shared, stack, count, 4)["status"]

    assert run() == 0
    assert run(src=(0, 2, 1)) == X and run(src=(0, 1 << 30, 1)) == X
    assert run(keep=(11, 7, 5)) == C and run(keep=(-1, 7, 5)) == C
    assert run(held=(13, 7)) == C and run(held=(10, -7), src=(0, 0, 0), keep=(10, 10, 10)) == C
    assert run(count=11, src=(0, 1, -1)) == Bk and run(count=-1, src=(0, 1, -1), keep=(8, 4, 0)) == Bk
    for x in (-1, 10):  # kept whole, kept in part, given back, taken
        assert run(table=((x, 1, 2), (3, 4, -9))) == Bk
        assert run(table=((0, 1, x), (3, 4, -9))) == Bk
        assert run(table=((0, 1, 2), (3, x, -9)), src=(0, -1, -1)) == Bk
        assert run(stack=(9, 8, 7, 6, x, 0, 0, 0, 0, 0)) == Bk


def test_a_full_stack_drops_what_is_given_back(ws):
    w = run_fork(ws, [-1], None, [8], [[1, 2]], [0] * 4, [0, 3, 0, 3], 3, 4)
    assert w["status"] == binding.GQA_DEV_BAD_BLOCK and w["free_count"][0] == 4


def test_random_steps_keep_every_block_once(ws):
    """Sixty steps of forks, ends and cuts in place of one another: afterwards, as
    after each, a block is either free once or held by as many tables as `shared` says."""
    r = np.random.default_rng(11)
    B, bs, mb = 24, 4, 10
    held, table, shared, stack, count = pool_of_requests(r, B, bs, mb, 60)
    for _ in range(60):
        src = r.integers(-1, B, B)
        keep = np.where(src < 0, 0, r.integers(0, held[np.maximum(src, 0)] + 1))
        w = run_fork(ws, src, keep, held, table, shared, stack, count, bs, True)
        assert w["status"] == 0
        held, table, shared, stack, count = (w["kv_lens"], w["block_table"], w["shared"], w["free_blocks"], int(w["free_count"][0]))
        seen = np.zeros(len(shared), int)
        for b in range(B):
            for j in range(-(-int(held[b]) // bs)):
                seen[table[b, j]] += 1
                if (j + 1) * bs > held[b]:
                    assert shared[table[b, j]] == 0
        free = stack[:count]
        assert len(set(free)) == count and not seen[free].any()
        assert ((seen == shared + 1) | ((seen == 0) & (shared == 0))).all()
        # grow on blocks of the stack, as a step does
        for b in range(B):
            have = -(-int(held[b]) // bs)
            grown = min(mb * bs, int(held[b]) + int(r.integers(0, 9)))
            need = -(-grown // bs) - have
            if need <= count:
                for i in range(need):
                    count -= 1
                    table[b, have + i] = stack[count]
                held[b] = grown


# ---------------------------------------------------------------- copies

def run_copy(ws, src, dst, rows, k, v):
    want_k, want_v, want = oracle.copy_blocks(src, dst, rows, *(bits(x if x.dim() == 5 else x[None]) for x in (k, v)))
    binding.gqa_attn_copy_blocks(i32(src), i32(dst), i32(rows), k, v, ws)
    assert (bits(k).reshape(want_k.shape) == want_k).all() and (bits(v).reshape(want_v.shape) == want_v).all()
    assert status(ws) == want
    return want


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,bs,layers,Hkv", [(1, 64, 28, 4), (7, 16, 3, 2), (60, 7, 2, 1), (3, 333, None, 8), (2, 1, 5, 5)])
def test_copies(ws, dtype, D, n, bs, layers, Hkv):
    r = np.random.default_rng(n)
    order = r.permutation(2 * n + 1)
    src, dst, rows = r.choice(order[:n], n), order[n:2 * n], r.integers(0, bs + 1, n)
    src = np.where(r.random(n) < 0.2, -1, src)
    shape = (2 * n + 1, Hkv, bs, D)
    k, v = (inputs.randn(shape if layers is None else (layers, *shape), s, dtype, DEV) for s in (1, 2))
    assert run_copy(ws, src, dst, rows, k, v) == 0
    assert run_copy(ws, src, dst, None, k, v) == 0


def test_copy_bad_input(ws):
    k, v = (inputs.randn((2, 6, 2, 8, 64), s, torch.bfloat16, DEV) for s in (1, 2))
    for src, dst, rows, want in (([6, 0], [1, 2], [8, 8], binding.GQA_DEV_BAD_BLOCK),
                                 ([1, 0], [6, 2], None, binding.GQA_DEV_BAD_BLOCK),
                                 ([1, 0], [-1, 2], None, binding.GQA_DEV_BAD_BLOCK),
                                 ([1, 0], [3, 2], [9, 8], binding.GQA_DEV_KVLEN_CLAMPED),
                                 ([1, 0], [3, 2], [-1, 8], binding.GQA_DEV_KVLEN_CLAMPED),
                                 ([1, -5], [1, -9], [9, -8], binding.GQA_DEV_KVLEN_CLAMPED), ([-1, -1], [3, 3], None, 0)):
        binding.gqa_attn_clear_device_status(ws)
        assert run_copy(ws, src, dst, rows, k, v) == want


def test_rows_past_32_bits(ws):
    """The far end of caches of more than 2^32 elements."""
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 20 GB")
    layers, n, Hkv, bs, D = 2, 33_000, 8, 64, 128
    k, v = (torch.zeros((layers, n, Hkv, bs, D), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    for x, s in ((k, 1), (v, 2)):
        x[:, n - 3:] = inputs.randn((layers, 3, Hkv, bs, D), s, torch.bfloat16, DEV)
    tail = [x[:, n - 3:].clone() for x in (k, v)]
    binding.gqa_attn_copy_blocks(i32([n - 1]), i32([n - 2]), i32([50]), k, v, ws)
    out = i32([0])
    binding.gqa_attn_compact_rows(i32([[2, 9]]), i32([2]), i32([10]), i32([64]), i32([[n - 3]]), k, v, out, ws)
    want = oracle.copy_blocks([2], [1], [50], *map(bits, tail))
    want = oracle.compact_rows([[2, 9]], [2], [10], [64], [[0]], *want[:2])
    assert (bits(k[:, n - 3:]) == want[0]).all() and (bits(v[:, n - 3:]) == want[1]).all() and ints(out) == [56]
    assert not k[:, :n - 3].any() and not v[:, :n - 3].any() and status(ws) == 0
