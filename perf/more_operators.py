"""Performance cases of verifying drafted tokens and of sharing a cache's pages.

Five operators, each with a plain form in elementary torch operations and the
call a program makes of the library:

  tables   ancestor masks and positions of a tree of drafted tokens from its
           parents (gqa_attn_tree_tables)
  tree     attention of the drafted tokens over the cache, dense and paged, with
           the tree's mask or as a chain (gqa_attn_decode_tree, _paged)
  compact  the accepted path's rows moved together in every layer's cache
           (gqa_attn_compact_rows)
  fork     block tables of requests that continue, fork, shorten or end, with
           shared whole blocks (gqa_attn_fork_tables)
  copy     the pages that forked requests do not share, copied in every layer
           (gqa_attn_copy_blocks)

Head geometries are the ones the library is benchmarked at: 14/2 heads of 64,
28/4 and 32/8 heads of 128.
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one request's small tree: the latency of a step
        {"name": "tables_B1_N26", "op": "tables", "B": 1, "N": 26, "Tq": 26, "ragged": False},
        # a batch of trees of 64 nodes, requests with fewer or none among them
        {"name": "tables_B256_N64", "op": "tables", "B": 256, "N": 64, "Tq": 64, "ragged": True},
        # eight drafted tokens of one short conversation, a dense cache
        {"name": "tree_B1_T8_L513_14x2x64", "op": "tree", "B": 1, "Hq": 14, "Hkv": 2, "D": 64, "N": 8, "Tq": 8, "L": 513,
         "ragged": False, "chain": False, "paged": False, "block": 64},
        # a few long conversations with large trees, odd sizes
        {"name": "tree_B4_T61_L16385_28x4x128", "op": "tree", "B": 4, "Hq": 28, "Hkv": 4, "D": 128, "N": 61, "Tq": 61,
         "L": 16385, "ragged": False, "chain": False, "paged": False, "block": 64},
        # a batch of requests of all lengths over a paged cache
        {"name": "tree_B32_T64_L8192_32x8x128", "op": "tree", "B": 32, "Hq": 32, "Hkv": 8, "D": 128, "N": 64, "Tq": 64,
         "L": 8192, "ragged": True, "chain": False, "paged": True, "block": 64},
        # a large batch that verifies up to four drafted tokens behind the last one
        {"name": "chain_B128_T5_L2048_32x8x128", "op": "tree", "B": 128, "Hq": 32, "Hkv": 8, "D": 128, "N": 5, "Tq": 5,
         "L": 2048, "ragged": True, "chain": True, "paged": True, "block": 64},
        # the accepted rows of one request in a model's 28 layers
        {"name": "compact_B1_N16_28layers_4x128", "op": "compact", "B": 1, "layers": 28, "Hkv": 4, "D": 128, "N": 16,
         "block": 64, "paged": True, "dtype": "bf16"},
        # those of a batch
        {"name": "compact_B128_N64_16layers_8x128", "op": "compact", "B": 128, "layers": 16, "Hkv": 8, "D": 128, "N": 64,
         "block": 64, "paged": True, "dtype": "bf16"},
        # a step of eight beams over one long prompt
        {"name": "fork_B8_L8192", "op": "fork", "B_in": 8, "B": 8, "block": 64, "L": 8192, "room": 64, "fresh": 0.1,
         "spare": 512},
        # a batch in which some samples end, some fork and drafted rows are given back
        {"name": "fork_B256_L8192", "op": "fork", "B_in": 256, "B": 256, "block": 64, "L": 8192, "room": 300,
         "fresh": 0.6, "spare": 1000},
        # one forked request's last page in a model's 28 layers
        {"name": "copy_n1_28layers_4x64x128", "op": "copy", "n": 1, "layers": 28, "Hkv": 4, "D": 128, "block": 64,
         "idle": 0, "dtype": "bf16"},
        # those of many requests forked at once, most of the list idle
        {"name": "copy_n256_16layers_8x64x128", "op": "copy", "n": 256, "layers": 16, "Hkv": 8, "D": 128, "block": 64,
         "idle": 160, "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tables", "tree", "tree", "tree", "compact", "fork", "copy"])
    Hq, Hkv, D = rng.choice([(14, 2, 64), (28, 4, 128), (32, 8, 128), (8, 8, 64), (16, 1, 128)])
    if op == "tables":
        N = _log_int(rng, 1, 200)
        return {"op": op, "B": _log_int(rng, 1, 400), "N": N, "Tq": rng.choice([N, N, max(1, N // 3)]),
                "ragged": rng.random() < 0.6}
    if op == "tree":
        B, N = _log_int(rng, 1, 100), _log_int(rng, 1, 160)
        Tq = rng.choice([N, N, N, max(1, N // 4)])
        L = N + _log_int(rng, 1, 16000)
        while 4.0 * B * L * Hq * Tq * D > 2e11 or B * Hkv * L * D > 2e8:
            L = N + (L - N) * 3 // 4
        return {"op": op, "B": B, "Hq": Hq, "Hkv": Hkv, "D": D, "N": N, "Tq": Tq, "L": L, "ragged": rng.random() < 0.6,
                "chain": rng.random() < 0.3, "paged": rng.random() < 0.5, "block": rng.choice([64, 128, 192])}
    if op == "compact":
        return {"op": op, "B": _log_int(rng, 1, 128), "layers": rng.randint(1, 16), "Hkv": Hkv, "D": D,
                "N": _log_int(rng, 2, 100), "block": rng.choice([16, 64, 128]), "paged": rng.random() < 0.7,
                "dtype": rng.choice(["bf16", "bf16", "f32"])}
    if op == "fork":
        B_in = _log_int(rng, 1, 300)
        return {"op": op, "B_in": B_in, "B": rng.choice([B_in, B_in, _log_int(rng, 1, 300)]),
                "block": rng.choice([16, 64, 128]), "L": _log_int(rng, 20, 8192), "room": rng.randint(0, 300),
                "fresh": rng.uniform(0, 1), "spare": _log_int(rng, 1, 3000)}
    return {"op": op, "n": _log_int(rng, 1, 100), "layers": rng.randint(1, 16), "Hkv": Hkv, "D": D,
            "block": rng.choice([16, 64, 128]), "idle": rng.randint(0, 20), "dtype": rng.choice(["bf16", "bf16", "f32"])}


# ---------------------------------------------------------------- inputs

def _randn(shape, dtype, g):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)


def _ints(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def _zeros(*shape):
    return torch.zeros(shape, dtype=torch.int32, device=DEV)


def _dtype(case):
    return torch.float32 if case.get("dtype") == "f32" else torch.bfloat16


def _words(N):
    return (N + 31) // 32


def _trees(r, B, N):
    """Parents of B random trees of N nodes: each node's is one before it, node 0
    and a few others begin at the last token of the cache."""
    p = np.floor(r.random((B, N)) * np.arange(N)).astype(np.int64)
    p[r.random((B, N)) < 0.03] = -1
    p[:, 0] = -1
    return p


def _ancestors(parents):
    """bool [B, N, N]: whether node j is node i itself or above it."""
    B, N = parents.shape
    a = np.zeros((B, N, N), dtype=bool)
    for i in range(N):
        p = parents[:, i]
        a[:, i] = np.where((p >= 0)[:, None], a[np.arange(B), np.maximum(p, 0)], False)
        a[:, i, i] = True
    return a


def _packed(bits):
    """int32 words of bool [..., N], bit j of a row in word j // 32."""
    n = bits.shape[-1]
    full = np.zeros(bits.shape[:-1] + (_words(n) * 32,), dtype=np.uint8)
    full[..., :n] = bits
    return np.packbits(full, axis=-1, bitorder="little").view(np.int32)


def _queries(r, case, nodes):
    """Nodes of each request and its queries, the last of these."""
    B, N, Tq = case["B"], case["N"], case["Tq"]
    if not case["ragged"]:
        return np.full(B, nodes), np.full(B, min(Tq, nodes))
    n = r.integers(0 if B > 2 else 1, nodes + 1, B)
    n[int(r.integers(0, B))] = nodes
    return n, np.minimum(n, Tq)


def _prepare_tables(case, seed):
    r = np.random.default_rng(seed)
    B, N, Tq = case["B"], case["N"], case["Tq"]
    n, q = _queries(r, case, N)
    starts = np.concatenate([[0], np.cumsum(q)])
    T = B * Tq
    kv = r.integers(0, 30000, B) + n
    return {"parents": _ints(_trees(r, B, N)), "tree_lens": _ints(n), "q_lens": _ints(q), "kv_lens": _ints(kv),
            "q_starts": _ints(starts), "mask": _zeros(B, Tq, _words(N)), "positions": _zeros(T), "Tq": Tq, "T": T}


def _prepare_tree(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    r = np.random.default_rng(seed)
    B, Hq, Hkv, D, N, Tq, L = (case[x] for x in ("B", "Hq", "Hkv", "D", "N", "Tq", "L"))
    dt = torch.bfloat16
    n, ql = _queries(r, case, N)
    if case["chain"]:
        n = ql
    lens = r.integers(N, L + 1, B) if case["ragged"] else np.full(B, L)
    lens[int(r.integers(0, B))] = L
    rows = _ancestors(_trees(r, B, N))
    bits = np.zeros((B, Tq, N), dtype=bool)
    at = (n - ql)[:, None] + np.arange(Tq)  # the node of each query
    ok = np.arange(Tq) < ql[:, None]
    bits[ok] = rows[np.nonzero(ok)[0], at[ok]]
    s = {"q": _randn((B, Hq, Tq, D), dt, g), "o": torch.zeros((B, Hq, Tq, D), dtype=dt, device=DEV), "lens": _ints(lens),
         "q_lens": _ints(ql), "tree_lens": None if case["chain"] else _ints(n), "L": L, "N": N,
         "mask": None if case["chain"] else _ints(_packed(bits)), "scale": D ** -0.5, "dims": (B, Hq, Hkv, D, Tq)}
    if case["paged"]:
        bs = case["block"]
        mb = -(-L // bs)
        n_pool = B * mb + 2
        s |= {"k": _randn((n_pool, Hkv, bs, D), dt, g), "v": _randn((n_pool, Hkv, bs, D), dt, g),
              "table": _ints(r.permutation(n_pool)[:B * mb].reshape(B, mb))}
    else:
        s |= {"k": _randn((B, Hkv, L, D), dt, g), "v": _randn((B, Hkv, L, D), dt, g), "table": None}
    return s


def _prepare_compact(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    r = np.random.default_rng(seed)
    B, NL, Hkv, D, N, bs = (case[x] for x in ("B", "layers", "Hkv", "D", "N", "block"))
    most = min(N, 10)
    keep = r.integers(1, most + 1, B)
    # node 0, then nodes of deeper and deeper levels: either the next ones or ones
    # behind all the places that the path moves to (so that a pass run again on
    # the same rows leaves the same)
    path = np.zeros((B, most), dtype=np.int64)
    for b in range(B):
        m = int(keep[b])
        near = int(r.integers(1, m + 1))  # the first ones are where they belong
        near = m if N - m < m - near else near
        path[b, :near] = np.arange(near)
        path[b, near:m] = np.sort(r.choice(np.arange(m, N), m - near, replace=False)) if m > near else []
        path[b, m:] = -1
    prior = r.integers(0, bs + 1, B)
    mb = -(-(bs + N) // bs)
    s = {"path": _ints(path), "keep": _ints(keep), "tree_lens": _ints(np.full(B, N)), "lens": _ints(prior + N),
         "lens_out": _zeros(B)}
    if case["paged"]:
        n_pool = B * mb + 2
        shape = (NL, n_pool, Hkv, bs, D)
        s["table"] = _ints(r.permutation(n_pool)[:B * mb].reshape(B, mb))
    else:
        shape = (NL, B, Hkv, bs + N, D)
        s["table"] = None
    s |= {"k": _randn(shape, _dtype(case), g), "v": _randn(shape, _dtype(case), g)}
    return s


def _prepare_fork(case, seed):
    r = np.random.default_rng(seed)
    B_in, B, bs, L = case["B_in"], case["B"], case["block"], case["L"]
    mb = -(-L // bs)
    # requests in families that share the whole blocks of their common prompt
    family = np.sort(r.integers(0, max(1, B_in // 4), B_in))
    common = r.integers(0, L + 1, B_in)[family] // bs  # whole blocks of the family's prompt
    held = np.maximum(common * bs, r.integers(0, L + 1, B_in))
    held = np.where(r.random(B_in) < 0.05, 0, np.minimum(held, L))
    have = -(-held // bs)
    j = np.arange(mb)
    mine = (j >= common[:, None]) & (j < have[:, None])
    shares = (j < common[:, None]) & (j < have[:, None])
    n_pool = int(max(1, B_in // 4)) * mb + B_in * mb + case["spare"]
    order = r.permutation(n_pool)
    table = np.where(shares, order[family[:, None] * mb + j], 0)
    table = np.where(mine, order[max(1, B_in // 4) * mb + np.arange(B_in)[:, None] * mb + j], table)
    holders = np.bincount(table[shares | mine], minlength=n_pool)
    stack = np.zeros(n_pool, dtype=np.int64)
    stack[:case["spare"]] = order[-case["spare"]:]
    # who continues whom: most the request before, some another one's fork, some none
    src = np.where(r.random(B) < case["fresh"], np.arange(B) % B_in, r.integers(0, B_in, B))
    src = np.where(r.random(B) < 0.05, -1, src)
    keep = np.maximum(held[np.maximum(src, 0)] - r.integers(0, case["room"] + 1, B), 0)
    keep = np.where(r.random(B) < 0.5, held[np.maximum(src, 0)], keep)
    return {"src": _ints(src), "keep": _ints(keep), "held": _ints(held), "table": _ints(table),
            "shared": _ints(np.maximum(holders - 1, 0)), "free": _ints(stack), "count": _ints([case["spare"]]), "bs": bs,
            "out": {"block_table": _zeros(B, mb), "kv_lens": _zeros(B), "shared": _zeros(n_pool), "free": _zeros(n_pool),
                    "free_count": _zeros(1), "copy_src": _zeros(B), "copy_dst": _zeros(B), "copy_rows": _zeros(B)}}


def _prepare_copy(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    r = np.random.default_rng(seed)
    n, NL, Hkv, D, bs = (case[x] for x in ("n", "layers", "Hkv", "D", "block"))
    live = max(1, n - case["idle"])
    n_src = max(1, live // 2)
    pool = live + n_src + 3
    order = r.permutation(pool)
    src, dst, rows = np.full(n, -1), np.full(n, -1), np.zeros(n, dtype=np.int64)
    at = np.sort(r.permutation(n)[:live])
    src[at], dst[at] = order[r.integers(0, n_src, live)], order[n_src:n_src + live]  # (some forked more than once)
    rows[at] = r.integers(1, bs + 1, live)
    shape = (NL, pool, Hkv, bs, D)
    return {"src": _ints(src), "dst": _ints(dst), "rows": _ints(rows), "k": _randn(shape, _dtype(case), g),
            "v": _randn(shape, _dtype(case), g)}


_PREPARE = {"tables": _prepare_tables, "tree": _prepare_tree, "compact": _prepare_compact, "fork": _prepare_fork,
            "copy": _prepare_copy}


def prepare(case, seed):
    return {"op": case["op"], **_PREPARE[case["op"]](case, seed)}


# ---------------------------------------------------------------- plain forms

def _plain_tables(s):
    parents = s["parents"].long()
    dev, (B, N), Tq = parents.device, parents.shape, s["Tq"]
    W = _words(N)
    node = torch.arange(N, device=dev)
    # ancestors: powers of the step to the parent (its distances doubled)
    reach = torch.eye(N, device=dev) + (parents[:, :, None] == node).float()
    steps = 1
    while steps < N:
        reach = (torch.bmm(reach, reach) > 0).float()
        steps *= 2
    n, q = s["tree_lens"].long(), s["q_lens"].long()
    i = torch.arange(Tq, device=dev)
    at = (n - q)[:, None] + i
    ok = i < q[:, None]
    rows = torch.gather(reach, 1, at.clamp(0, N - 1)[:, :, None].expand(B, Tq, N))
    full = torch.zeros((B, Tq, W * 32), device=dev)
    full[:, :, :N] = rows
    word = (full.view(B, Tq, W, 32).long() << torch.arange(32, device=dev)).sum(-1)
    word = torch.where(word >= 2 ** 31, word - 2 ** 32, word)
    mask = torch.where(ok[:, :, None], word.int(), s["mask"])
    pos = (s["kv_lens"].long() - n)[:, None] + rows.sum(-1).long() - 1
    t = (s["q_starts"][:B].long()[:, None] + i)[ok]
    positions = s["positions"].index_put((t,), pos[ok].int())
    return {"mask": mask, "positions": positions}


def _cache_rows(s):
    """K and V [B, Hkv, L, D] of a tree case as they are stored."""
    if s["table"] is None:
        return s["k"], s["v"]
    rows = lambda pool: pool[s["table"].long()].transpose(1, 2).flatten(2, 3)[:, :, :s["L"]]  # noqa: E731
    return rows(s["k"]), rows(s["v"])


def _visible(s):
    """bool [B, Tq, L]: the keys of each query."""
    Tq, L, dev = s["dims"][4], s["L"], s["q"].device
    lens, ql = s["lens"].long()[:, None, None], s["q_lens"].long()[:, None, None]
    j, i = torch.arange(L, device=dev)[None, None, :], torch.arange(Tq, device=dev)[None, :, None]
    if s["mask"] is None:
        return (j <= lens - ql + i) & (j < lens)
    c = j - (lens - s["tree_lens"].long()[:, None, None])  # drafted row of the key
    words = s["mask"][:, :, None, :].expand(-1, -1, 1, -1).squeeze(2)
    bit = torch.gather(words, 2, (c >> 5).clamp(0, words.shape[2] - 1).expand(-1, Tq, -1)) >> (c & 31).int()
    return ((c < 0) | ((bit & 1) > 0)) & (j < lens)


def _plain_tree(s):
    B, Hq, Hkv, D, Tq = s["dims"]
    n = Hq // Hkv
    k, v = (x.float() for x in _cache_rows(s))
    q = s["q"].float().view(B, Hkv, n * Tq, D)
    x = torch.matmul(q, k.transpose(2, 3)) * s["scale"]
    x = x.view(B, Hkv, n, Tq, -1).masked_fill(~_visible(s)[:, None, None], -float("inf"))
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(m == -float("inf"), 0.0, m))
    l = e.sum(-1, keepdim=True)
    o = torch.matmul(e.view(B, Hkv, n * Tq, -1), v).view(B, Hkv, n, Tq, D)
    o = torch.where(l > 0, o / l, 0.0).reshape(B, Hq, Tq, D).to(s["q"].dtype)
    live = torch.arange(Tq, device=q.device) < s["q_lens"].long()[:, None]
    return torch.where(live[:, None, :, None], o, s["o"])


def _plain_compact(s):
    path, keep = s["path"].long(), s["keep"].long()
    k = torch.arange(path.shape[1], device=path.device)
    base = (s["lens"] - s["tree_lens"]).long()
    ok = k < keep[:, None]
    b = torch.arange(path.shape[0], device=path.device)[:, None].expand_as(ok)[ok]
    frm, to = (base[:, None] + path)[ok], (base[:, None] + k)[ok]
    bs = s["k"].shape[3]
    at = (lambda r: (b, r)) if s["table"] is None else (lambda r: (s["table"].long()[b, r // bs], r % bs))
    (fb, fr), (tb, tr) = at(frm), at(to)
    s["k"][:, tb, :, tr] = s["k"][:, fb, :, fr]
    s["v"][:, tb, :, tr] = s["v"][:, fb, :, fr]
    return {"k": s["k"], "v": s["v"], "kv_lens": (base + keep).int()}


def _plain_fork(s):
    o, dev = s["out"], s["src"].device
    src, bs, table = s["src"].long(), s["bs"], s["table"].long()
    B, (B_in, mb), pool = src.shape[0], table.shape, s["shared"].shape[0]
    held, count = s["held"].long(), s["count"].long()[0]
    none = src < 0
    sc = src.clamp(min=0)
    keep = torch.where(none, 0, torch.minimum(s["keep"].long(), held[sc]))
    b, j = torch.arange(B, device=dev), torch.arange(mb, device=dev)
    # the owner of an old request: of those that continue it, the one that keeps most, the first of equals
    rank = torch.where(none, -1, keep * B + (B - 1 - b))
    best = torch.full((B_in,), -1, dtype=torch.long, device=dev).scatter_reduce(0, sc, rank, "amax")
    owner = ~none & (best[sc] == rank)
    whole, rest = keep // bs, keep % bs
    last = table[sc, whole.clamp(max=mb - 1)]  # the block that is kept in part
    stays = owner & (rest > 0) & (s["shared"].long()[last] == 0)
    wants = ~none & (rest > 0) & ~stays
    nth = wants.long().cumsum(0) - 1
    copies = wants & (nth < count)
    cut = wants & ~copies
    rest = torch.where(cut, 0, rest)
    taken = s["free"].long()[(count - 1 - nth).clamp(0, pool - 1)]
    n_taken = copies.sum()
    mine = torch.where(j[None, :] == whole[:, None], torch.where(copies, taken, last)[:, None], table[sc])
    kept = j[None, :] < (whole + (rest > 0))[:, None]
    table_out = torch.where(kept, mine, o["block_table"].long())
    # holders: one more for each whole block of another than the owner, one less for each that the owner does not keep
    by = torch.zeros(B_in, dtype=torch.long, device=dev).scatter_reduce(0, sc, torch.where(owner, whole + stays, 0), "amax")
    gone = (j[None, :] >= by[:, None]) & (j[None, :] < ((held + bs - 1) // bs)[:, None])
    more = ~owner[:, None] & ~none[:, None] & (j[None, :] < whole[:, None])
    shared = s["shared"].long() + torch.bincount(table[sc][more], minlength=pool) - torch.bincount(table[gone], minlength=pool)
    # blocks that nobody holds go onto the stack, in the order of the tables
    flat = torch.arange(B_in * mb, device=dev).view(B_in, mb)
    first = torch.full((pool,), B_in * mb, dtype=torch.long, device=dev).scatter_reduce(0, table[gone], flat[gone], "amin")
    pushed = table[gone & (shared[table] < 0) & (first[table] == flat)]
    at = count - n_taken + torch.arange(pushed.shape[0], device=dev)
    free = s["free"].long().index_put((at,), pushed)
    out = {"block_table": table_out, "kv_lens": whole * bs + rest, "shared": shared.clamp(min=0), "free": free,
           "free_count": (count - n_taken + pushed.shape[0]).reshape(1), "copy_src": torch.where(copies, last, -1),
           "copy_dst": torch.where(copies, taken, -1), "copy_rows": torch.where(copies, rest, 0)}
    return {k: v.int() for k, v in out.items()}


def _plain_copy(s):
    live = s["src"] >= 0
    src, dst, rows = s["src"][live].long(), s["dst"][live].long(), s["rows"][live]
    take = (torch.arange(s["k"].shape[3], device=src.device) < rows[:, None])[None, :, None, :, None]
    s["k"][:, dst] = torch.where(take, s["k"][:, src], s["k"][:, dst])
    s["v"][:, dst] = torch.where(take, s["v"][:, src], s["v"][:, dst])
    return {"k": s["k"], "v": s["v"]}


# ---------------------------------------------------------------- the library's calls

def _scratch(s, n):
    """A call's workspace, allocated once and kept, as a program does."""
    if "ws" not in s:
        s["ws"] = torch.zeros(n, dtype=torch.uint8, device=DEV)
    return s["ws"]


def _own_tables(s):
    from gqa_attention_kv_decode_gb300 import binding
    binding.gqa_attn_tree_tables(s["parents"], s["tree_lens"], s["q_lens"], s["kv_lens"], s["q_starts"], s["mask"],
                                 s["positions"], _scratch(s, 256))
    return {"mask": s["mask"], "positions": s["positions"]}


def _own_tree(s):
    from gqa_attention_kv_decode_gb300 import binding
    B, Hq, Hkv, D, Tq = s["dims"]
    if "ws" not in s:
        _scratch(s, binding.gqa_attn_decode_tree_workspace_size(B, Hq, Hkv, D, Tq, s["L"]))
    if s["table"] is None:
        binding.gqa_attn_decode_tree(s["q"], s["k"], s["v"], s["mask"], s["q_lens"], s["tree_lens"], s["lens"], s["o"],
                                     s["scale"], s["ws"])
    else:
        binding.gqa_attn_decode_tree_paged(s["q"], s["k"], s["v"], s["table"], s["mask"], s["q_lens"], s["tree_lens"],
                                           s["lens"], s["o"], s["scale"], s["ws"], s["L"])
    return s["o"]


def _own_compact(s):
    from gqa_attention_kv_decode_gb300 import binding
    binding.gqa_attn_compact_rows(s["path"], s["keep"], s["tree_lens"], s["lens"], s["table"], s["k"], s["v"],
                                  s["lens_out"], _scratch(s, 256))
    return {"k": s["k"], "v": s["v"], "kv_lens": s["lens_out"]}


def _own_fork(s):
    from gqa_attention_kv_decode_gb300 import binding
    o = s["out"]
    binding.gqa_attn_fork_tables(s["src"], s["keep"], s["held"], s["table"], s["shared"], s["free"], s["count"],
                                 o["block_table"], o["kv_lens"], o["shared"], o["free"], o["free_count"], o["copy_src"],
                                 o["copy_dst"], o["copy_rows"], s["bs"], _scratch(s, 256))
    return o


def _own_copy(s):
    from gqa_attention_kv_decode_gb300 import binding
    binding.gqa_attn_copy_blocks(s["src"], s["dst"], s["rows"], s["k"], s["v"], _scratch(s, 256))
    return {"k": s["k"], "v": s["v"]}


def run(state):
    if own:
        return {"tables": _own_tables, "tree": _own_tree, "compact": _own_compact, "fork": _own_fork,
                "copy": _own_copy}[state["op"]](state)
    return {"tables": _plain_tables, "tree": _plain_tree, "compact": _plain_compact, "fork": _plain_fork,
            "copy": _plain_copy}[state["op"]](state)


# ---------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op == "tables":
        half = 0.5 if case["ragged"] else 1.0
        nodes, queries = case["B"] * case["N"] * half, case["B"] * case["Tq"] * half
        # a parent a node; the words of a query's mask, its position; four lengths a request
        return {"bytes": 4.0 * (nodes + queries * (_words(case["N"]) + 1) + 4 * case["B"]), "flops": 0.0}
    if op == "tree":
        B, Hq, Hkv, D, N, Tq, L = (case[x] for x in ("B", "Hq", "Hkv", "D", "N", "Tq", "L"))
        keys = B * ((N + L) / 2 if case["ragged"] else L)
        queries = B * Tq * (0.5 if case["ragged"] else 1.0)
        return {"bytes": 4.0 * Hkv * D * keys + 4.0 * queries * Hq * D, "flops": 4.0 * Hq * D * keys * queries / B}
    e = 4 if case.get("dtype") == "f32" else 2
    if op == "compact":
        # half of the kept rows behind the first move, in K and V of every layer
        moved = case["B"] * (min(case["N"], 10) - 1) / 4
        return {"bytes": 4.0 * moved * case["layers"] * case["Hkv"] * case["D"] * e + 16.0 * case["B"], "flops": 0.0}
    if op == "fork":
        mb = -(-case["L"] // case["block"])
        pool = max(1, case["B_in"] // 4) * mb + case["B_in"] * mb + case["spare"]
        # the kept tables read and written (half of them in the mean), holders and stack in and out
        return {"bytes": 4.0 * (case["B"] * mb + 4 * pool + 6 * case["B"] + case["B_in"]), "flops": 0.0}
    live = max(1, case["n"] - case["idle"])
    return {"bytes": 4.0 * live * (case["block"] + 1) / 2 * case["layers"] * case["Hkv"] * case["D"] * e, "flops": 0.0}


# ---------------------------------------------------------------- in 64 bits

def _np(t):
    return t.cpu().numpy().astype(np.int64)


def _exact_tables(case, s):
    parents, n, q, kv, starts = (_np(s[x]) for x in ("parents", "tree_lens", "q_lens", "kv_lens", "q_starts"))
    mask, positions = _np(s["mask"]), _np(s["positions"])
    for b in range(case["B"]):
        for i in range(q[b]):
            node, above = n[b] - q[b] + i, []
            while node >= 0:
                above.append(int(node))
                node = parents[b, node]
            bits = sum(1 << x for x in above)
            for w in range(mask.shape[2]):
                x = bits >> (32 * w) & 0xffffffff
                mask[b, i, w] = x - (1 << 32) if x >> 31 else x
            positions[starts[b] + i] = kv[b] - n[b] + len(above) - 1
    return {"mask": torch.from_numpy(mask.astype(np.int32)), "positions": torch.from_numpy(positions.astype(np.int32))}


def _exact_tree(case, s):
    B, Hq, Hkv, D, Tq = s["dims"]
    lens, ql = _np(s["lens"]), _np(s["q_lens"])
    out = s["o"].double()
    for b in range(B):
        m, L = int(ql[b]), int(lens[b])
        if m == 0:
            continue
        if s["table"] is None:
            k, v = s["k"][b, :, :L].double(), s["v"][b, :, :L].double()
        else:
            bs = case["block"]
            ids = s["table"][b, :-(-L // bs)].long()
            k, v = (x[ids].transpose(0, 1).reshape(Hkv, -1, D)[:, :L].double() for x in (s["k"], s["v"]))
        see = np.ones((m, L), dtype=bool)
        if s["mask"] is None:
            see[:, L - m:] = np.tril(see[:, L - m:])
        else:
            n = int(_np(s["tree_lens"])[b])
            words = s["mask"][b, :m].cpu().numpy().view(np.uint8).reshape(m, -1)
            see[:, L - n:] = np.unpackbits(words, axis=1, bitorder="little")[:, :n] > 0
        hide = torch.from_numpy(~see).to(DEV)
        for g in range(Hkv):
            h = slice(g * (Hq // Hkv), (g + 1) * (Hq // Hkv))
            w = torch.softmax((s["q"][b, h, :m].double() @ k[g].T * s["scale"]).masked_fill(hide, -math.inf), -1)
            out[b, h, :m] = w @ v[g]
    return out


def _exact_compact(case, s):
    path, keep, n, lens = (_np(s[x]) for x in ("path", "keep", "tree_lens", "lens"))
    table = None if s["table"] is None else _np(s["table"])
    out, rows = {}, s["k"].shape[3]
    frm, to = [], []
    for b in range(case["B"]):
        base = int(lens[b] - n[b])
        for k in range(int(keep[b])):
            for at, r in ((frm, base + int(path[b, k])), (to, base + k)):
                at.append((b if table is None else int(table[b, r // rows])) * rows + r % rows)
    frm, to = torch.tensor(frm, device=DEV), torch.tensor(to, device=DEV)
    for name in ("k", "v"):
        flat = s[name].double().transpose(2, 3).contiguous()  # [layers, blocks, rows, heads, D]
        view = flat.view(flat.shape[0], -1, *flat.shape[3:])
        view.index_copy_(1, to, view.index_select(1, frm))
        out[name] = flat.transpose(2, 3).contiguous()
    out["kv_lens"] = torch.from_numpy((lens - n + keep).astype(np.int32))
    return out


def _exact_fork(case, s):
    src, keep, held, table, shared, stack = (_np(s[x]) for x in ("src", "keep", "held", "table", "shared", "free"))
    bs, B, B_in = s["bs"], case["B"], case["B_in"]
    out = {k: _np(v) for k, v in s["out"].items()}
    top = int(_np(s["count"])[0])
    takers = [[b for b in range(B) if src[b] == a] for a in range(B_in)]
    keep = [0 if src[b] < 0 else min(int(keep[b]), int(held[src[b]])) for b in range(B)]
    owner = [max(t, key=lambda b: (keep[b], -b)) if t else None for t in takers]
    delta = np.zeros(shared.size, dtype=np.int64)
    kept_by_owner = [0] * B_in
    out["copy_src"][:], out["copy_dst"][:], out["copy_rows"][:] = -1, -1, 0
    for b in range(B):
        a, n = int(src[b]), keep[b]
        out["kv_lens"][b] = n
        if a < 0:
            continue
        whole, rest = divmod(n, bs)
        out["block_table"][b, :whole] = table[a, :whole]
        if owner[a] != b:
            for x in table[a, :whole]:
                delta[x] += 1
        else:
            kept_by_owner[a] = whole
        if rest:
            x = table[a, whole]
            if owner[a] == b and shared[x] == 0:
                kept_by_owner[a] += 1
                out["block_table"][b, whole] = x
            elif top > 0:
                top -= 1
                out["block_table"][b, whole] = stack[top]
                out["copy_src"][b], out["copy_dst"][b], out["copy_rows"][b] = x, stack[top], rest
            else:
                out["kv_lens"][b] = whole * bs
    gone = [int(table[a, j]) for a in range(B_in) for j in range(kept_by_owner[a], -(-int(held[a]) // bs))]
    for x in gone:
        delta[x] -= 1
    now = shared + delta
    free = stack.copy()
    for x in dict.fromkeys(gone):
        if now[x] < 0:
            free[top] = x
            top += 1
    out["shared"], out["free"], out["free_count"] = np.maximum(now, 0), free, np.array([top])
    return {k: torch.from_numpy(np.asarray(v).astype(np.int32)) for k, v in out.items()}


def _exact_copy(case, s):
    src, dst, rows = (_np(s[x]) for x in ("src", "dst", "rows"))
    out = {}
    for name in ("k", "v"):
        c = s[name].double()
        for i in np.nonzero(src >= 0)[0]:
            c[:, dst[i], :, :rows[i]] = c[:, src[i], :, :rows[i]]
        out[name] = c
    return out


def exact(case, seed):
    return {"tables": _exact_tables, "tree": _exact_tree, "compact": _exact_compact, "fork": _exact_fork,
            "copy": _exact_copy}[case["op"]](case, prepare(case, seed))
