"""Plain oracle of a serving step's other operations (test infrastructure).

  * ``step_tables``: block tables, slot map and lengths of one step, request by
    request, with Python lists for the free stack;
  * ``rope_append``: per-head RMS norm, rotary rotation and the scatter of Q,
    K and V, in float64;
  * ``attention_shared_prefix``: every request attends the shared prefix rows
    followed by its own, by the attention definition on the concatenated keys.

Everything is numpy; nothing here is used by the product path.
"""

from __future__ import annotations

import numpy as np

from .gqa_oracle import attention

CLAMPED, EMPTY, BAD_BLOCK, OUT_OF_BLOCKS, BAD_SLOT, BAD_POSITION = 1, 2, 8, 16, 32, 64


def step_tables(prior_lens, new_lens, T, block_size, q_rows, block_table=None, free_blocks=None, free_count=None):
    """One step's tables.  Returns a dict of int32 arrays (block_table,
    free_blocks and free_count only for a paged cache) and ``status``."""
    prior_lens, new_lens = np.asarray(prior_lens, dtype=np.int64), np.asarray(new_lens, dtype=np.int64)
    B = len(prior_lens)
    paged = block_table is not None
    status = 0
    if paged:
        table = np.array(block_table, dtype=np.int64)
        stack = np.array(free_blocks, dtype=np.int64)
        pool = len(stack)
        cap = table.shape[1] * block_size
        top = int(free_count)
        if not 0 <= top <= pool:
            status |= BAD_BLOCK
            top = min(max(top, 0), pool)
    else:
        cap = block_size

    def blocks(n):
        return -(-n // block_size)

    prior = np.clip(prior_lens, 0, cap)
    if (prior != prior_lens).any():
        status |= CLAMPED

    # finished requests give their blocks back
    if paged:
        for b in range(B):
            if new_lens[b] < 0:
                for i in range(blocks(int(prior[b]))):
                    blk = table[b, i]
                    if not 0 <= blk < pool:
                        status |= BAD_BLOCK
                    if top < pool:
                        stack[top] = blk
                        top += 1
                    else:
                        status |= BAD_BLOCK

    kv, ql = np.zeros(B, np.int64), np.zeros(B, np.int64)
    starts = np.zeros(B + 1, np.int64)
    pos, slots, q_slots = np.zeros(T, np.int64), np.full(T, -1), np.full(T, -1)
    avail, wanted, first = (top if paged else 0), 0, 0
    for b in range(B):
        n = int(new_lens[b])
        starts[b + 1] = min(first + max(n, 0), T)
        if n < 0:
            continue
        kv[b] = prior[b]
        at, first = first, first + n
        if first > T or n > q_rows or prior[b] + n > cap:
            status |= CLAMPED
            continue
        if paged:
            have = blocks(int(prior[b]))
            need = blocks(int(prior[b]) + n) - have
            wanted += need
            if need > 0 and wanted > avail:
                status |= OUT_OF_BLOCKS
                continue
            for i in range(need):
                top -= 1
                blk = stack[top]
                if not 0 <= blk < pool:
                    status |= BAD_BLOCK
                table[b, have + i] = blk
        kv[b], ql[b] = prior[b] + n, n
        for i in range(n):
            p = int(prior[b]) + i
            blk = int(table[b, p // block_size]) if paged else b
            if paged and not 0 <= blk < pool:
                status |= BAD_BLOCK
                continue
            pos[at + i] = p
            slots[at + i] = blk * block_size + (p % block_size if paged else p)
            q_slots[at + i] = b * q_rows + i
    out = {"kv_lens": kv, "q_lens": ql, "q_starts": starts, "positions": pos, "slots": slots, "q_slots": q_slots}
    if paged:
        out |= {"block_table": table, "free_blocks": stack, "free_count": np.array([top])}
    out = {k: v.astype(np.int32) for k, v in out.items()}
    out["status"] = status
    return out


def rms_norm(x, weight, eps):
    """x [..., D] scaled to unit mean square, times weight; x if there is none."""
    x = np.asarray(x, dtype=np.float64)
    if weight is None:
        return x
    return x / np.sqrt((x * x).mean(axis=-1, keepdims=True) + eps) * np.asarray(weight, dtype=np.float64)


def rotate(x, cos, sin, adjacent):
    """Rotates the first 2 * cos.shape[-1] dims of x [T, H, D] by the angles of
    each token (cos, sin [T, R / 2])."""
    y = np.array(x, dtype=np.float64)
    R = 2 * cos.shape[-1]
    for i in range(R // 2):
        a, b = (2 * i, 2 * i + 1) if adjacent else (i, i + R // 2)
        c, s = cos[:, i, None], sin[:, i, None]
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def rope_append(q, k, v, q_weight, k_weight, eps, cos_sin, positions, slots, q_slots, q_out, k_cache, v_cache,
                adjacent):
    """(q_out, k_cache, v_cache, status) after the tokens were written, float64."""
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    T = q.shape[0]
    slots = np.asarray(slots, dtype=np.int64)
    q_slots = np.arange(T) if q_slots is None else np.asarray(q_slots, dtype=np.int64)
    q, k = rms_norm(q, q_weight, eps), rms_norm(k, k_weight, eps)
    bad = np.zeros(T, dtype=bool)
    status = 0
    out = [np.array(x, dtype=np.float64) for x in (q_out, k_cache, v_cache)]
    n_q, n_kv = out[0].shape[0] * out[0].shape[2], out[1].shape[0] * out[1].shape[2]
    if (slots >= n_kv).any() or (q_slots >= n_q).any():
        status |= BAD_SLOT
    slots, q_slots = np.where(slots >= n_kv, -1, slots), np.where(q_slots >= n_q, -1, q_slots)
    if cos_sin is not None:
        cos_sin = np.asarray(cos_sin, dtype=np.float64)
        positions = np.asarray(positions, dtype=np.int64)
        bad = ((positions < 0) | (positions >= cos_sin.shape[0])) & ((slots >= 0) | (q_slots >= 0))
        if bad.any():
            status |= BAD_POSITION
        cs = cos_sin[np.clip(positions, 0, cos_sin.shape[0] - 1)]
        R = cs.shape[1]
        q, k = (rotate(x, cs[:, :R // 2], cs[:, R // 2:], adjacent) for x in (q, k))
    for t in range(T):
        if bad[t]:
            continue
        if q_slots[t] >= 0:
            g, r = divmod(int(q_slots[t]), out[0].shape[2])
            out[0][g, :, r] = q[t]
        if slots[t] >= 0:
            g, r = divmod(int(slots[t]), out[1].shape[2])
            out[1][g, :, r] = k[t]
            out[2][g, :, r] = v[t]
    return (*out, status)


def attention_shared_prefix(q, k_prefix, v_prefix, k, v, kv_lens, scale=None):
    """q [B, Hq, 1, D]; k_prefix, v_prefix [Hkv, P, D] seen by every request
    before its own rows [0, kv_lens[b]) of k, v [B, Hkv, S, D]."""
    q = np.asarray(q, dtype=np.float64)
    out = np.zeros_like(q)
    for b in range(q.shape[0]):
        L = int(kv_lens[b])
        kk = np.concatenate([np.asarray(k_prefix, dtype=np.float64), np.asarray(k[b][:, :L], dtype=np.float64)], 1)
        vv = np.concatenate([np.asarray(v_prefix, dtype=np.float64), np.asarray(v[b][:, :L], dtype=np.float64)], 1)
        if kk.shape[1] == 0:
            continue  # no key: zeros
        out[b] = attention(q[b:b + 1], kk[None], vv[None], scale=scale)["o"][0]
    return out
