"""Plain oracle of verifying drafted tokens and of sharing a cache's pages (test
infrastructure).

  * ``tree_tables``: ancestor masks and positions, node by node;
  * ``attention_tree``: every query attends the rows before the drafted ones and
    the drafted rows that its mask names, by the attention definition;
  * ``compact_rows``, ``copy_blocks``: rows copied one by one;
  * ``fork_tables``: new requests one after the other, holders counted in a dict.

Everything is numpy and Python; nothing here is used by the product path.
"""

from __future__ import annotations

import numpy as np

CLAMPED, EMPTY, BAD_BLOCK, OUT_OF_BLOCKS, BAD_INDEX = 1, 2, 8, 16, 128


def _clamp(x, lo, hi):
    return min(max(int(x), lo), hi)


def tree_tables(parents, tree_lens, q_lens, mask, kv_lens=None, q_starts=None, positions=None):
    """(mask, positions, status) after the call; mask int32 [B, Tq, words] and
    positions [T] (or None) are what stood there before."""
    parents, mask = np.asarray(parents), np.array(mask, dtype=np.int32)
    positions = None if positions is None else np.array(positions, dtype=np.int32)
    B, N = parents.shape
    Tq, W = mask.shape[1:]
    status = 0
    for b in range(B):
        n = _clamp(tree_lens[b], 0, N)
        most = min(Tq, n)
        q = most if q_lens is None else _clamp(q_lens[b], 0, most)
        if n != tree_lens[b] or (q_lens is not None and q != q_lens[b]):
            status |= CLAMPED
        if positions is not None and kv_lens[b] < n:
            status |= CLAMPED
        above = []
        for i in range(n):
            p = int(parents[b, i])
            if p >= i or p < -1:
                status |= BAD_INDEX
                p = -1
            above.append((above[p] if p >= 0 else set()) | {i})
        for i in range(q):
            node = n - q + i
            for w in range(W):
                word = sum(1 << (c - 32 * w) for c in above[node] if 32 * w <= c < 32 * w + 32)
                mask[b, i, w] = np.uint32(word).astype(np.int32)
            if positions is not None:
                t = int(q_starts[b]) + i
                if 0 <= t < len(positions):
                    positions[t] = max(int(kv_lens[b]) - n, 0) + len(above[node]) - 1
    return mask, positions, status


def tree_visible(mask, Tq, q_len, tree_len, kv_len):
    """bool [q_len, kv_len] of one request; mask int32 [Tq, words] or None (a chain)."""
    see = np.ones((q_len, kv_len), dtype=bool)
    for i in range(q_len):
        if mask is None:
            see[i, kv_len - q_len + i + 1:] = False
        else:
            for c in range(tree_len):
                see[i, kv_len - tree_len + c] = (int(mask[i, c // 32]) >> (c % 32)) & 1
    return see


def attention_tree(q, k, v, mask, q_lens, tree_lens, kv_lens, scale, before):
    """(o, status): q [B, Hq, Tq, D], k and v [B, Hkv, S, D]; `before` is what o
    holds, of which the rows past the lengths stay."""
    q, o = np.asarray(q, dtype=np.float64), np.array(before, dtype=np.float64)
    B, Hq, Tq, _ = q.shape
    Hkv, S = k.shape[1], k.shape[2]
    status = 0
    for b in range(B):
        L = _clamp(kv_lens[b], 0, S)
        want_q = Tq if q_lens is None else q_lens[b]
        ql = _clamp(want_q, 0, min(Tq, L))
        want_n = 0 if mask is None else ql if tree_lens is None else tree_lens[b]
        n = _clamp(want_n, 0, min(32 * mask.shape[2], L) if mask is not None else 0)
        if L != kv_lens[b] or ql != want_q or n != want_n:
            status |= CLAMPED
        see = tree_visible(None if mask is None else mask[b], Tq, ql, n, L)
        if ql and not see.any(axis=1).all():
            status |= EMPTY
        for h in range(Hq):
            g = h // (Hq // Hkv)
            kk, vv = (np.asarray(x[b, g, :L], dtype=np.float64) for x in (k, v))
            s = np.where(see, q[b, h, :ql] @ kk.T * scale, -np.inf)
            m = s.max(axis=1, initial=-np.inf, keepdims=True)
            w = np.exp(s - np.where(np.isfinite(m), m, 0.0))
            total = w.sum(axis=1, keepdims=True)
            o[b, h, :ql] = np.where(total > 0, (w @ vv) / np.where(total > 0, total, 1.0), 0.0)
    return o, status


def compact_rows(path, n_keep, tree_lens, kv_lens, table, k_cache, v_cache):
    """(k_cache, v_cache, kv_lens_out, status); caches [layers, blocks, Hkv, rows, D]."""
    k, v = np.array(k_cache), np.array(v_cache)
    pool, bs = k.shape[1], k.shape[3]
    B, P = np.asarray(path).shape
    cap = bs if table is None else np.asarray(table).shape[1] * bs
    out, status = np.zeros(B, np.int32), 0
    for b in range(B):
        L = _clamp(kv_lens[b], 0, cap)
        n = _clamp(tree_lens[b], 0, L)
        keep = _clamp(n_keep[b], 0, min(P, n))
        if (L, n, keep) != (kv_lens[b], tree_lens[b], n_keep[b]):
            status |= CLAMPED
        nodes = [int(c) for c in path[b][:keep]]
        base = L - n
        out[b] = base
        if any(c >= n or c < 0 for c in nodes) or nodes != sorted(set(nodes)):
            status |= BAD_INDEX
            continue
        out[b] = base + keep
        moves = []
        for i, c in enumerate(nodes):
            if c == i:
                continue
            at = []
            for r in (base + c, base + i):
                blk, row = (b, r) if table is None else (int(table[b][r // bs]), r % bs)
                if not 0 <= blk < pool:
                    status |= BAD_BLOCK
                at.append((blk, row))
            if all(0 <= blk < pool for blk, _ in at):
                moves.append(at)
        for x in (k, v):
            rows = [x[:, s, :, r].copy() for (s, r), _ in moves]
            for (_, (d, r)), row in zip(moves, rows):
                x[:, d, :, r] = row
    return k, v, out, status


def fork_tables(src, keep_lens, held_lens, table, shared, free_blocks, free_count, table_out, block_size):
    """A dict of the outputs (table_out: what stood there before) and ``status``."""
    table, out = np.asarray(table), np.array(table_out, dtype=np.int64)
    B_in, mb = table.shape
    pool, B, cap = len(shared), len(src), mb * block_size
    status = 0
    held = [_clamp(h, 0, cap) for h in held_lens]
    if held != [int(h) for h in held_lens]:
        status |= CLAMPED
    count = _clamp(free_count, 0, pool)
    if count != free_count:
        status |= BAD_BLOCK

    def valid(x):
        nonlocal status
        if not 0 <= x < pool:
            status |= BAD_BLOCK
        return 0 <= x < pool

    keep, came = [], []
    for b in range(B):
        s = int(src[b])
        if s >= B_in:
            status |= BAD_INDEX
            s = -1
        came.append(max(s, -1))
        want = 0 if s < 0 else held[s] if keep_lens is None else int(keep_lens[b])
        keep.append(_clamp(want, 0, held[s]) if s >= 0 else 0)
        if s >= 0 and keep[-1] != want:
            status |= CLAMPED
    owner = {}
    for b in range(B):
        if came[b] >= 0 and (came[b] not in owner or keep[b] > keep[owner[came[b]]]):
            owner[came[b]] = b
    holders = {x: int(n) + 1 for x, n in enumerate(shared)}
    stack, top = [int(x) for x in free_blocks], count
    stay = [0] * B_in
    lens, copies = np.zeros(B, np.int64), []
    for b in range(B):
        s = came[b]
        copies.append((-1, -1, 0))
        if s < 0:
            continue
        whole, rest = divmod(keep[b], block_size)
        lens[b] = whole * block_size
        for j in range(whole):
            x = int(table[s][j])
            out[b][j] = x
            if valid(x) and owner[s] != b:
                holders[x] += 1
        if owner[s] == b:
            stay[s] = whole
        if rest:
            x = int(table[s][whole])
            ok = valid(x)
            if owner[s] == b and (not ok or shared[x] == 0):
                out[b][whole], stay[s] = x, whole + 1
                lens[b] += rest
            elif top > 0:
                top -= 1
                valid(stack[top])
                out[b][whole] = stack[top]
                copies[-1] = (x, stack[top], rest)
                lens[b] += rest
            else:
                status |= OUT_OF_BLOCKS
    gone = []
    for s in range(B_in):
        for j in range(stay[s], -(-held[s] // block_size)):
            x = int(table[s][j])
            if valid(x):
                holders[x] -= 1
                gone.append(x)
    for x in dict.fromkeys(gone):
        if holders[x] <= 0:
            holders[x] = 1
            if top < pool:
                stack[top] = x
                top += 1
            else:
                status |= BAD_BLOCK
    res = {"block_table": out, "kv_lens": lens, "shared": np.array([holders[x] - 1 for x in range(pool)]),
           "free_blocks": np.array(stack), "free_count": np.array([top])}
    res |= {name: np.array([c[i] for c in copies]) for i, name in enumerate(("copy_src", "copy_dst", "copy_rows"))}
    return {k: v.astype(np.int32) for k, v in res.items()} | {"status": status}


def copy_blocks(src, dst, rows, k_cache, v_cache):
    """(k_cache, v_cache, status); caches [layers, blocks, Hkv, block_size, D]."""
    k, v = np.array(k_cache), np.array(v_cache)
    pool, bs = k.shape[1], k.shape[3]
    status = 0
    for i, s in enumerate(src):
        if s < 0:
            continue
        n = bs if rows is None else _clamp(rows[i], 0, bs)
        if rows is not None and n != rows[i]:
            status |= CLAMPED
        if s >= pool or not 0 <= dst[i] < pool:
            status |= BAD_BLOCK
            continue
        for x in (k, v):
            x[:, dst[i], :, :n] = x[:, s, :, :n]
    return k, v, status
