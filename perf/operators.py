"""Performance cases of the operators of a serving step around the KV cache.

Three operators, each with a plain form in elementary torch operations and the
call a program makes of the library:

  tables   block tables, slot map, positions and lengths of one step, built on
           the GPU from the requests' lengths (gqa_attn_step_tables)
  append   per-head norm of Q and K, rotary rotation, Q to the attention's
           layout, K and V into the cache (gqa_attn_rope_append)
  prefix   single-token decode of a batch whose requests share their first
           keys (gqa_attn_decode_shared_prefix, dense and paged)

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
        # one decode step of a running batch: a token a request, a few requests
        # idle or finished, tables of up to 8192 keys in blocks of 64
        {"name": "tables_decode_B64", "op": "tables", "B": 64, "block": 64, "max_blocks": 128, "chunk": 1,
         "chunked": 0, "done": 4, "idle": 3, "room": 64, "dense": False},
        # prefill chunks of 512 beside running decodes, with too few free
        # blocks for all of them
        {"name": "tables_mixed_B256", "op": "tables", "B": 256, "block": 64, "max_blocks": 128, "chunk": 512,
         "chunked": 16, "done": 11, "idle": 5, "room": 100, "dense": False},
        # the first step of many prompts
        {"name": "tables_prompts_B96", "op": "tables", "B": 96, "block": 128, "max_blocks": 64, "chunk": 2049,
         "chunked": 96, "done": 0, "idle": 0, "room": 2000, "dense": False},
        # one token of one request: the latency of a step
        {"name": "append_T1_14x2x64", "op": "append", "T": 1, "pad": 0, "Hq": 14, "Hkv": 2, "D": 64, "dtype": "bf16",
         "rot": 64, "pairs": "half", "norm": False, "block": 2048, "q_rows": 1, "far": 2048},
        # a decode step of 61 requests padded to the 64 of its captured graph
        {"name": "append_T64_32x8x128", "op": "append", "T": 64, "pad": 3, "Hq": 32, "Hkv": 8, "D": 128,
         "dtype": "bf16", "rot": 128, "pairs": "half", "norm": True, "block": 64, "q_rows": 1, "far": 8192},
        # an fp32 cache, neighbouring dims rotated, half of each head
        {"name": "append_T2049_14x2x64_f32", "op": "append", "T": 2049, "pad": 0, "Hq": 14, "Hkv": 2, "D": 64,
         "dtype": "f32", "rot": 32, "pairs": "adjacent", "norm": True, "block": 128, "q_rows": 2049, "far": 131072},
        # a whole prompt, no norms
        {"name": "append_T4097_28x4x128", "op": "append", "T": 4097, "pad": 0, "Hq": 28, "Hkv": 4, "D": 128,
         "dtype": "bf16", "rot": 128, "pairs": "half", "norm": False, "block": 4352, "q_rows": 4097, "far": 4097},
        # a large prefill step of many chunks
        {"name": "append_T16384_32x8x128", "op": "append", "T": 16384, "pad": 0, "Hq": 32, "Hkv": 8, "D": 128,
         "dtype": "bf16", "rot": 128, "pairs": "half", "norm": True, "block": 64, "q_rows": 512, "far": 32768},
        # a few requests behind a short instruction
        {"name": "prefix_B4_P513_14x2x64", "op": "prefix", "B": 4, "Hq": 14, "Hkv": 2, "D": 64, "P": 513, "room": 0,
         "S": 128, "paged": False, "block": 64},
        # samples of one long prompt, an odd length in a larger buffer
        {"name": "prefix_B16_P4097_28x4x128", "op": "prefix", "B": 16, "Hq": 28, "Hkv": 4, "D": 128, "P": 4097,
         "room": 255, "S": 512, "paged": False, "block": 64},
        # a batch of questions about one long document
        {"name": "prefix_B64_P32768_32x8x128", "op": "prefix", "B": 64, "Hq": 32, "Hkv": 8, "D": 128, "P": 32768,
         "room": 0, "S": 1024, "paged": True, "block": 64},
        # a large batch, where the prefix is bound by the products
        {"name": "prefix_B256_P16384_32x8x128", "op": "prefix", "B": 256, "Hq": 32, "Hkv": 8, "D": 128, "P": 16384,
         "room": 0, "S": 512, "paged": True, "block": 64},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tables", "append", "append", "prefix", "prefix"])
    Hq, Hkv, D = rng.choice([(14, 2, 64), (28, 4, 128), (32, 8, 128), (8, 8, 64), (16, 1, 128)])
    if op == "tables":
        B = _log_int(rng, 1, 512)
        chunk = _log_int(rng, 1, 2049)
        chunked = rng.randint(0, min(B, 96))
        dense = rng.random() < 0.25
        return {"op": op, "B": B, "block": rng.choice([64, 128, 192, 256]), "max_blocks": rng.randint(33, 128),
                "chunk": chunk, "chunked": chunked, "done": rng.randint(0, (B - chunked) // 4),
                "idle": rng.randint(0, (B - chunked) // 4), "room": _log_int(rng, 8, 4000), "dense": dense}
    if op == "append":
        T = _log_int(rng, 1, 12000)
        dtype = rng.choice(["bf16", "bf16", "f32"])
        q_rows = rng.choice([1, 1, 37, 512, T])
        return {"op": op, "T": T, "pad": rng.randint(0, T // 4), "Hq": Hq, "Hkv": Hkv, "D": D, "dtype": dtype,
                "rot": 16 * rng.randint(1, D // 16), "pairs": rng.choice(["half", "half", "adjacent"]),
                "norm": rng.random() < 0.6, "block": rng.choice([64, 128, 320, 1000]), "q_rows": q_rows,
                "far": _log_int(rng, 64, 131072)}
    B = _log_int(rng, 1, 200)
    P = _log_int(rng, 1, 16384)
    return {"op": op, "B": B, "Hq": Hq, "Hkv": Hkv, "D": D, "P": P, "room": rng.choice([0, 0, 1, 200, 4000]),
            "S": _log_int(rng, 1, 600), "paged": rng.random() < 0.5, "block": rng.choice([64, 128, 192])}


# ---------------------------------------------------------------- inputs

def _randn(shape, dtype, g):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)


def _ints(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def _prepare_tables(case, seed):
    r = np.random.default_rng(seed)
    B, bs, mb, chunk = case["B"], case["block"], case["max_blocks"], case["chunk"]
    cap = bs * mb
    kind = np.zeros(B, dtype=np.int64)  # 0 decode, 1 chunk, 2 done, 3 idle
    kind[:case["chunked"]] = 1
    kind[case["chunked"]:case["chunked"] + case["done"]] = 2
    kind[case["chunked"] + case["done"]:case["chunked"] + case["done"] + case["idle"]] = 3
    r.shuffle(kind)
    new = np.where(kind == 0, 1, np.where(kind == 1, r.integers(1, chunk + 1, B), np.where(kind == 2, -1, 0)))
    most = np.maximum(cap - np.maximum(new, 0), 0)
    prior = r.integers(0, most + 1)
    prior[(kind == 1) & (r.random(B) < 0.5)] = 0  # half of the chunks begin a prompt
    T = (B - case["chunked"]) + case["chunked"] * chunk  # the rows of the step's token buffers
    s = {"prior": _ints(prior), "new": _ints(new), "bs": cap if case["dense"] else bs, "T": T, "q_rows": chunk,
         "dense": case["dense"], "B": B}
    if not case["dense"]:
        have = -(-prior // bs)
        n_pool = B * mb + case["room"]  # (the blocks in neither a table nor the stack are held elsewhere)
        order = r.permutation(n_pool)
        table = np.zeros((B, mb), dtype=np.int64)
        at = np.concatenate([[0], np.cumsum(have)])
        for b in range(B):
            table[b, :have[b]] = order[at[b]:at[b + 1]]
        free = np.zeros(n_pool, dtype=np.int64)
        free[:case["room"]] = order[at[-1]:at[-1] + case["room"]]
        s |= {"table": _ints(table), "free": _ints(free), "count": _ints([case["room"]]), "n_pool": n_pool}
    s["out"] = {"kv_lens": torch.empty(B, dtype=torch.int32, device=DEV),
                "q_lens": torch.empty(B, dtype=torch.int32, device=DEV),
                "q_starts": torch.empty(B + 1, dtype=torch.int32, device=DEV),
                "positions": torch.empty(T, dtype=torch.int32, device=DEV),
                "slots": torch.empty(T, dtype=torch.int32, device=DEV),
                "q_slots": torch.empty(T, dtype=torch.int32, device=DEV)}
    if not case["dense"]:
        s["out"]["free_count"] = torch.empty(1, dtype=torch.int32, device=DEV)
    return s


def _rope_table(n, rot):
    """fp32 [n, rot]: cos of the rot / 2 angles of each position, then their sin."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
    a = torch.arange(n, dtype=torch.float64, device=DEV)[:, None] * inv[None, :]
    return torch.cat([a.cos(), a.sin()], dim=1).float()


def _prepare_append(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    r = np.random.default_rng(seed)
    T, Hq, Hkv, D = case["T"], case["Hq"], case["Hkv"], case["D"]
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    # the projections' output: the q, k and v heads of a token side by side
    qkv = _randn((T, (Hq + 2 * Hkv) * D), dt, g)
    q, k, v = (x.unflatten(1, (-1, D)) for x in qkv.split([Hq * D, Hkv * D, Hkv * D], dim=1))
    bs, q_rows = case["block"], case["q_rows"]
    n_blocks = -(-T // bs) + 2
    live = T - case["pad"]
    # runs of consecutive rows, as chunks and decodes leave them: blocks in any order
    rows = np.arange(n_blocks * bs).reshape(n_blocks, bs)[r.permutation(n_blocks)].reshape(-1)
    slots = np.full(T, -1)
    slots[:live] = rows[:live]
    start = int(r.integers(0, max(1, case["far"] - T)))
    positions = np.where(np.arange(T) < live, (start + np.arange(T)) % case["far"], 0)
    groups = -(-T // q_rows)
    q_slots = np.where(np.arange(T) < live, np.arange(T), -1)
    s = {"q": q, "k": k, "v": v, "slots": _ints(slots), "positions": _ints(positions), "q_slots": _ints(q_slots),
         "rot": case["rot"], "adjacent": case["pairs"] == "adjacent", "eps": 1e-6, "wq": None, "wk": None,
         "table": _rope_table(case["far"], case["rot"]),
         "q_out": _randn((groups, Hq, q_rows, D), dt, g),
         "k_cache": _randn((n_blocks, Hkv, bs, D), dt, g), "v_cache": _randn((n_blocks, Hkv, bs, D), dt, g)}
    if case["norm"]:
        s["wq"] = (1.0 + 0.2 * torch.randn(D, generator=g, device=DEV)).to(dt)
        s["wk"] = (1.0 + 0.2 * torch.randn(D, generator=g, device=DEV)).to(dt)
    return s


def _prepare_prefix(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    r = np.random.default_rng(seed)
    B, Hq, Hkv, D, P, S = (case[x] for x in ("B", "Hq", "Hkv", "D", "P", "S"))
    dt = torch.bfloat16
    lens = r.integers(0 if B > 2 else 1, S + 1, B)
    lens[int(r.integers(0, B))] = S
    s = {"q": _randn((B, Hq, 1, D), dt, g), "lens": _ints(lens), "p_len": _ints([P]), "P": P, "P_cap": P + case["room"],
         "S": S, "scale": D ** -0.5, "paged": case["paged"], "o": torch.empty((B, Hq, 1, D), dtype=dt, device=DEV),
         "dims": (B, Hq, Hkv, D)}
    if case["paged"]:
        bs = case["block"]
        np_blocks, ns_blocks = -(-(P + case["room"]) // bs), -(-S // bs)
        n = np_blocks + B * ns_blocks + 2
        order = r.permutation(n)
        s |= {"kp": _randn((n, Hkv, bs, D), dt, g), "vp": _randn((n, Hkv, bs, D), dt, g),
              "p_table": _ints(order[:np_blocks]),
              "table": _ints(order[np_blocks:np_blocks + B * ns_blocks].reshape(B, ns_blocks))}
    else:
        s |= {"kp": _randn((Hkv, P + case["room"], D), dt, g), "vp": _randn((Hkv, P + case["room"], D), dt, g),
              "k": _randn((B, Hkv, S, D), dt, g), "v": _randn((B, Hkv, S, D), dt, g)}
    return s


def prepare(case, seed):
    return {"op": case["op"], **{"tables": _prepare_tables, "append": _prepare_append,
                                 "prefix": _prepare_prefix}[case["op"]](case, seed)}


# ---------------------------------------------------------------- plain forms

def _plain_tables(s):
    dev, B, T, bs, q_rows = s["prior"].device, s["B"], s["T"], s["bs"], s["q_rows"]
    mb = 1 if s["dense"] else s["table"].shape[1]
    cap = mb * bs
    prior = s["prior"].long().clamp(0, cap)
    release = s["new"] < 0
    n = s["new"].long().clamp(min=0)
    end = n.cumsum(0)
    start = end - n
    fits = ~release & (end <= T) & (prior + n <= cap) & (n <= q_rows)
    if s["dense"]:
        ok = fits
        table = torch.arange(B, device=dev)[:, None]
    else:
        pool = s["n_pool"]
        have = (prior + bs - 1) // bs
        count = s["count"].long().clamp(0, pool)
        j = torch.arange(mb, device=dev)[None, :]
        # finished requests' blocks go on top of the stack, in request order
        freed = torch.where(release, have, 0)
        f_at = count + (freed.cumsum(0) - freed)[:, None] + j
        f_ok = (j < freed[:, None]) & (f_at < pool)
        stack = torch.cat([s["free"].long(), torch.zeros(1, dtype=torch.long, device=dev)])
        stack = stack.scatter(0, torch.where(f_ok, f_at, pool).reshape(-1), s["table"].long().reshape(-1))[:pool]
        avail = (count + freed.sum()).clamp(max=pool)
        # and the growing requests take theirs from it
        need = torch.where(fits, (prior + n + bs - 1) // bs - have, 0)
        upto = need.cumsum(0)
        ok = fits & ((need == 0) | (upto <= avail))
        taken = torch.where(ok & (need > 0), upto, 0).max()
        k = (upto - need)[:, None] + j - have[:, None]
        grows = ok[:, None] & (j >= have[:, None]) & (j < (have + need)[:, None])
        table = torch.where(grows, stack[(avail - 1 - k).clamp(0, pool - 1)], s["table"].long())
    granted = torch.where(ok, n, 0)
    t = torch.arange(T, device=dev)
    b = torch.searchsorted(end, t, right=True).clamp(max=B - 1)
    i = t - start[b]
    live = ok[b] & (t < end[-1])
    pos = torch.where(live, prior[b] + i, 0)
    slot = table[b, (pos // bs).clamp(max=mb - 1)] * bs + pos % bs
    out = {"kv_lens": torch.where(release, 0, prior + granted), "q_lens": granted,
           "q_starts": torch.cat([torch.zeros(1, dtype=torch.long, device=dev), end]).clamp(max=T),
           "positions": pos, "slots": torch.where(live, slot, -1), "q_slots": torch.where(live, b * q_rows + i, -1)}
    if not s["dense"]:
        out |= {"block_table": table, "free_blocks": stack, "free_count": (avail - taken).reshape(1)}
    return {k: v.int() for k, v in out.items()}


def _rotate(y, cos, sin, adjacent):
    """Rotates the first 2 * cos.shape[-1] dims of y [T, H, D]."""
    h = cos.shape[-1]
    a, b = (y[..., 0:2 * h:2], y[..., 1:2 * h:2]) if adjacent else (y[..., :h], y[..., h:2 * h])
    ra, rb = a * cos - b * sin, b * cos + a * sin
    r = torch.stack([ra, rb], dim=-1).flatten(-2) if adjacent else torch.cat([ra, rb], dim=-1)
    return torch.cat([r, y[..., 2 * h:]], dim=-1)


def _plain_append(s):
    def norm(x, w):
        x = x.float()
        return x if w is None else x * (x.square().mean(-1, keepdim=True) + s["eps"]).rsqrt() * w.float()

    cs = s["table"][s["positions"].long()][:, None, :]
    cos, sin = cs[..., :s["rot"] // 2], cs[..., s["rot"] // 2:]
    q = _rotate(norm(s["q"], s["wq"]), cos, sin, s["adjacent"]).to(s["q"].dtype)
    k = _rotate(norm(s["k"], s["wk"]), cos, sin, s["adjacent"]).to(s["k"].dtype)

    def put(cache, slots, x):
        keep = slots >= 0
        at = slots[keep].long()
        cache[at // cache.shape[2], :, at % cache.shape[2]] = x[keep]

    put(s["q_out"], s["q_slots"], q)
    put(s["k_cache"], s["slots"], k)
    put(s["v_cache"], s["slots"], s["v"])
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _gathered(s):
    """(prefix K, V [Hkv, P_cap, D], suffix K, V [B, Hkv, S, D]) of a prefix case, as they are stored."""
    if not s["paged"]:
        return s["kp"], s["vp"], s["k"], s["v"]
    def rows(pool, table, n):  # [..., blocks] -> [..., Hkv, n, D]
        x = pool[table.long()].transpose(-4, -3)
        return x.flatten(-3, -2)[..., :n, :]
    return (rows(s["kp"], s["p_table"], s["P_cap"]), rows(s["vp"], s["p_table"], s["P_cap"]),
            rows(s["kp"], s["table"], s["S"]), rows(s["vp"], s["table"], s["S"]))


def _plain_prefix(s):
    B, Hq, Hkv, D = s["dims"]
    n = Hq // Hkv
    kp, vp, k, v = (x.float() for x in _gathered(s))
    q = s["q"].float().view(B, Hkv, n, D)
    inf = float("inf")
    sp = torch.matmul(q.transpose(0, 1).reshape(Hkv, B * n, D), kp.transpose(1, 2)) * s["scale"]
    sp = sp.masked_fill(torch.arange(s["P_cap"], device=q.device) >= s["p_len"], -inf)
    ss = torch.matmul(q, k.transpose(2, 3)) * s["scale"]
    ss = ss.masked_fill(torch.arange(s["S"], device=q.device) >= s["lens"][:, None, None, None], -inf)
    mp = sp.amax(-1).view(Hkv, B, n).transpose(0, 1)
    m = torch.maximum(mp, ss.amax(-1))
    m = torch.where(m == -inf, 0.0, m)
    ep = torch.exp(sp - m.transpose(0, 1).reshape(Hkv, B * n, 1))
    es = torch.exp(ss - m[..., None])
    o = torch.matmul(ep, vp).view(Hkv, B, n, D).transpose(0, 1) + torch.matmul(es, v)
    l = ep.sum(-1).view(Hkv, B, n).transpose(0, 1) + es.sum(-1)
    o = torch.where(l[..., None] > 0, o / l[..., None], 0.0)
    return o.reshape(B, Hq, 1, D).to(s["q"].dtype)


# ---------------------------------------------------------------- the library's calls

def _scratch(s, n):
    """A call's workspace, allocated once and kept, as a program does."""
    if "ws" not in s:
        s["ws"] = torch.zeros(n, dtype=torch.uint8, device=DEV)
    return s["ws"]


def _own_tables(s):
    from gqa_attention_kv_decode_gb300 import binding
    o = s["out"]
    binding.gqa_attn_step_tables(s["prior"], s["new"], s.get("table"), s.get("free"), s.get("count"), o["kv_lens"],
                                 o["q_lens"], o["q_starts"], o["positions"], o["slots"], o["q_slots"],
                                 o.get("free_count"), s["bs"], s["q_rows"], _scratch(s, 256))
    return o if s["dense"] else {**o, "block_table": s["table"], "free_blocks": s["free"]}


def _own_append(s):
    from gqa_attention_kv_decode_gb300 import binding
    binding.gqa_attn_rope_append(s["q"], s["k"], s["v"], s["wq"], s["wk"], s["eps"], s["table"], s["positions"],
                                 s["slots"], s["q_slots"], s["q_out"], s["k_cache"], s["v_cache"], s["adjacent"],
                                 _scratch(s, 256))
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_prefix(s):
    from gqa_attention_kv_decode_gb300 import binding
    B, Hq, Hkv, D = s["dims"]
    if "ws" not in s:
        _scratch(s, binding.gqa_attn_decode_shared_prefix_workspace_size(B, Hq, Hkv, D, s["P_cap"], s["S"]))
    if s["paged"]:
        binding.gqa_attn_decode_shared_prefix_paged(s["q"], s["kp"], s["vp"], s["p_table"], s["p_len"], s["table"],
                                                    s["lens"], s["o"], s["scale"], s["ws"], s["P_cap"], s["S"])
    else:
        binding.gqa_attn_decode_shared_prefix(s["q"], s["kp"], s["vp"], s["p_len"], s["k"], s["v"], s["lens"], s["o"],
                                              s["scale"], s["ws"])
    return s["o"]


def run(state):
    if own:
        return {"tables": _own_tables, "append": _own_append, "prefix": _own_prefix}[state["op"]](state)
    return {"tables": _plain_tables, "append": _plain_append, "prefix": _plain_prefix}[state["op"]](state)


# ---------------------------------------------------------------- work

def work(case):
    if case["op"] == "tables":
        B, grows = case["B"], case["B"] - case["done"] - case["idle"]
        tokens = (B - case["chunked"]) + case["chunked"] * case["chunk"]
        new_blocks = 0 if case["dense"] else case["chunked"] * case["chunk"] // (2 * case["block"]) + grows // case["block"]
        # lengths in, lengths and starts out, three words a token, one table
        # entry a growing request, and a new block's id read and written
        return {"bytes": 4.0 * (2 * B + 3 * B + 1 + 3 * tokens + grows + 2 * new_blocks + 2), "flops": 0.0}
    if case["op"] == "append":
        e = 2 if case["dtype"] == "bf16" else 4
        live, heads = case["T"] - case["pad"], case["Hq"] + 2 * case["Hkv"]
        normed = (case["Hq"] + case["Hkv"]) * case["D"]
        return {"bytes": live * (2.0 * heads * case["D"] * e + min(1.0, case["far"] / case["T"]) * case["rot"] * 4)
                + 12.0 * case["T"] + (2.0 * case["D"] * e if case["norm"] else 0.0),
                "flops": live * ((4.0 * normed if case["norm"] else 0.0)
                                 + 3.0 * (case["Hq"] + case["Hkv"]) * case["rot"])}
    B, Hq, Hkv, D, P, S = (case[x] for x in ("B", "Hq", "Hkv", "D", "P", "S"))
    suffix = B * (S + 1) / 2
    return {"bytes": 4.0 * Hkv * D * (P + suffix) + 4.0 * B * Hq * D, "flops": 4.0 * Hq * D * (B * P + suffix)}


# ---------------------------------------------------------------- in 64 bits

def _exact_tables(case, s):
    g = {k: (v.cpu().numpy().astype(np.int64) if isinstance(v, torch.Tensor) else v) for k, v in s.items() if k != "out"}
    B, T, bs, rows, dense = s["B"], s["T"], s["bs"], s["q_rows"], s["dense"]
    table = np.arange(B)[:, None] if dense else g["table"].copy()
    free = [] if dense else list(g["free"][:int(g["count"][0])])
    stack = None if dense else g["free"].copy()
    cap = bs * table.shape[1]
    if not dense:
        for b in range(B):
            if g["new"][b] < 0:
                free += [int(x) for x in table[b, :-(-int(g["prior"][b]) // bs)]]
        stack[:len(free)] = free
    kv, ql, starts = np.zeros(B, np.int64), np.zeros(B, np.int64), np.zeros(B + 1, np.int64)
    pos, slot, qslot = np.zeros(T, np.int64), np.full(T, -1), np.full(T, -1)
    at, dry = 0, False
    for b in range(B):
        prior, n = int(g["prior"][b]), int(g["new"][b])
        if n < 0:
            starts[b + 1] = at
            continue
        first, at = at, at + n
        starts[b + 1] = min(at, T)
        kv[b] = prior
        if at > T or prior + n > cap or n > rows:
            continue
        if not dense:
            have, want = -(-prior // bs), -(-(prior + n) // bs)
            if want > have and (dry or want - have > len(free)):
                dry = True
                continue
            for i in range(have, want):
                table[b, i] = free.pop()
        kv[b], ql[b] = prior + n, n
        p = prior + np.arange(n)
        pos[first:at], slot[first:at], qslot[first:at] = p, table[b, p // bs] * bs + p % bs, b * rows + np.arange(n)
    out = {"kv_lens": kv, "q_lens": ql, "q_starts": starts, "positions": pos, "slots": slot, "q_slots": qslot}
    if not dense:
        out |= {"block_table": table, "free_blocks": stack, "free_count": np.array([len(free)])}
    return {k: torch.from_numpy(v.astype(np.int32)) for k, v in out.items()}


def _exact_append(case, s):
    half = case["rot"] // 2
    ang = s["table"].double()[s["positions"].long()]
    turn = torch.complex(ang[:, :half], ang[:, half:])[:, None]

    def head(x, w):
        x = x.double()
        if w is not None:
            x = x / ((x * x).sum(-1, keepdim=True) / case["D"] + s["eps"]).sqrt() * w.double()
        r = x[..., :2 * half]
        z = torch.complex(r[..., 0::2], r[..., 1::2]) if s["adjacent"] else torch.complex(r[..., :half], r[..., half:])
        z = z * turn
        r = torch.stack([z.real, z.imag], -1).flatten(-2) if s["adjacent"] else torch.cat([z.real, z.imag], -1)
        return torch.cat([r, x[..., 2 * half:]], -1)

    out = {}
    for name, at, x in (("q", "q_slots", head(s["q"], s["wq"])), ("k_cache", "slots", head(s["k"], s["wk"])),
                        ("v_cache", "slots", s["v"].double())):
        dst = s["q_out" if name == "q" else name].double().transpose(1, 2).contiguous()  # [n, rows, H, D]
        flat = dst.flatten(0, 1)
        live = s[at] >= 0
        flat[s[at][live].long()] = x[live]
        out[name] = flat.view(dst.shape).transpose(1, 2).contiguous()
    return out


def _exact_prefix(case, s):
    B, Hq, Hkv, D = s["dims"]
    kp, vp, k, v = _gathered(s)
    kp, vp = kp[:, :case["P"]].double(), vp[:, :case["P"]].double()
    n = Hq // Hkv
    out = torch.empty((B, Hq, D), dtype=torch.float64, device=DEV)
    lens = s["lens"].tolist()
    for b in range(B):
        kk = torch.cat([kp, k[b, :, :lens[b]].double()], 1)
        vv = torch.cat([vp, v[b, :, :lens[b]].double()], 1)
        w = torch.softmax(s["q"][b].double().view(Hkv, n, D) @ kk.transpose(1, 2) * s["scale"], -1)
        out[b] = (w @ vv).view(Hq, D)
    return out.view(B, Hq, 1, D)


def exact(case, seed):
    return {"tables": _exact_tables, "append": _exact_append, "prefix": _exact_prefix}[case["op"]](case,
                                                                                                prepare(case, seed))
