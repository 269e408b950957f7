"""The operators of a serving step together, as they are used: step tables,
norm-rotate-append, then attention over the cache they filled.

The reference keeps every request's normed, rotated keys and values as the
oracle computes them, rounds them once to the cache's type, and attends in
fp64.  The cache rows the GPU wrote may differ from these by one rounding (the
append's fp32 arithmetic against fp64, see tests/test_rope_append_gpu.py), so
the oracle attends the rows the GPU wrote, which are compared with the
reference's first: within one step of the type (2^-8 of the value), plus what
cancels in a rotation (76 * 2^-24 of the terms, below 2^-14 here).
"""

import threading

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


def ints(n):
    return torch.empty(n, dtype=torch.int32, device=DEV)


def ulp_close(got, ref):
    return (np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -14).all()


class Model:
    """One layer's weights, and the projections of every token of every request."""

    def __init__(self, Hq, Hkv, D, adjacent, max_pos, seed):
        self.Hq, self.Hkv, self.D, self.adjacent, self.seed = Hq, Hkv, D, adjacent, seed
        self.wq = (1 + 0.2 * inputs.randn((D,), seed, torch.float32, DEV)).to(BF16)
        self.wk = (1 + 0.2 * inputs.randn((D,), seed + 1, torch.float32, DEV)).to(BF16)
        self.cs = binding.rope_table(max_pos, D)
        self.eps = 1e-6

    def project(self, T, step):
        return inputs.randn((T, (self.Hq + 2 * self.Hkv) * self.D), 7000 + 97 * self.seed + step, BF16, DEV)

    def views(self, x):
        Hq, Hkv, D = self.Hq, self.Hkv, self.D
        return (y.unflatten(1, (-1, D)) for y in x.split([Hq * D, Hkv * D, Hkv * D], dim=1))

    def keys(self, x, positions):
        """The oracle's rotated K rows [T, Hkv, D] and V rows of projections x."""
        _, k, v = self.views(x)
        cs = f64(self.cs)[positions]
        k = oracle.rotate(oracle.rms_norm(f64(k), f64(self.wk), self.eps), cs[:, :self.D // 2], cs[:, self.D // 2:],
                          self.adjacent)
        return k, f64(v)


@pytest.mark.parametrize("Hq,Hkv,D,adjacent", [(32, 8, 128, False), (14, 2, 64, True)])
def test_paged_steps_in_one_graph(Hq, Hkv, D, adjacent):
    """A captured step (tables, append, paged decode), replayed while requests
    start, grow across block borders, pause and finish."""
    B, bs, mb, pool, T = 6, 64, 5, 24, 6
    m = Model(Hq, Hkv, D, adjacent, bs * mb, 3)
    kc = torch.full((pool, Hkv, bs, D), float("nan"), dtype=BF16, device=DEV)
    vc = torch.full_like(kc, float("nan"))
    lens, table = i32([0] * B), torch.zeros((B, mb), dtype=torch.int32, device=DEV)
    stack, count = i32(np.random.default_rng(0).permutation(pool)), i32([pool])
    new, q_lens, q_starts = i32([0] * B), ints(B), ints(B + 1)
    pos, slots, q_slots = ints(T), ints(T), ints(T)
    x = m.project(T, 0)
    q, k, v = m.views(x)
    q_out = torch.zeros((B, Hq, 1, D), dtype=BF16, device=DEV)
    o = torch.zeros_like(q_out)
    ws = binding.decode_workspace(B, Hq, Hkv, D, bs * mb, binding.GQA_BF16, DEV)

    def step():
        binding.gqa_attn_step_tables(lens, new, table, stack, count, lens, q_lens, q_starts, pos, slots, q_slots,
                                     count, bs, 1, ws)
        binding.gqa_attn_rope_append(q, k, v, m.wq, m.wk, m.eps, m.cs, pos, slots, q_slots, q_out, kc, vc,
                                     m.adjacent, ws)
        binding.gqa_attn_decode_paged(q_out, None, None, kc, vc, table, lens, o, D ** -0.5, ws, bs * mb)

    saved = [t.clone() for t in (lens, table, stack, count)]
    step()  # one-time kernel setup, outside the capture
    for t, s in zip((lens, table, stack, count), saved):
        t.copy_(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    binding.gqa_attn_clear_device_status(ws)
    r = np.random.default_rng(1)
    seen = [([], []) for _ in range(B)]
    for n in range(140):
        kinds = np.where(r.random(B) < 0.9, 1, 0)
        if n % 35 == 34:
            kinds[int(r.integers(0, B))] = -1
        new.copy_(i32(kinds))
        x.copy_(m.project(T, n))
        graph.replay()
        torch.cuda.synchronize()
        at = 0
        kk, vv = m.keys(x, np.array([len(seen[b][0]) for b in range(B) if kinds[b] == 1] + [0] * T)[:T])
        for b in range(B):
            if kinds[b] < 0:
                seen[b] = ([], [])
            elif kinds[b] == 1:
                seen[b][0].append(kk[at])
                seen[b][1].append(vv[at])
                at += 1
        L = [len(s[0]) for s in seen]
        assert lens.tolist() == L
        if n % 20 == 19 or n > 136:
            rows_k, rows_v = kc[table.long()], vc[table.long()]  # [B, mb, Hkv, bs, D]
            for b in range(B):
                if L[b] == 0 or kinds[b] != 1:
                    continue
                gk = f64(rows_k[b].transpose(0, 1).reshape(Hkv, mb * bs, D)[:, :L[b]])
                gv = f64(rows_v[b].transpose(0, 1).reshape(Hkv, mb * bs, D)[:, :L[b]])
                assert ulp_close(gk, np.stack(seen[b][0], 1)), (n, b)
                np.testing.assert_array_equal(gv, np.stack(seen[b][1], 1))
                ref = oracle.attention(f64(q_out[b:b + 1]), gk[None], gv[None], scale=D ** -0.5)["o"]
                parity.check(f64(o[b:b + 1]), ref, "bf16", f"step {n}, request {b}")
    status = binding.gqa_attn_read_device_status(ws)
    assert status & ~binding.GQA_DEV_EMPTY_REQUEST == 0


def test_prompts_then_decode_on_a_dense_cache():
    """Chunks of prompts into a dense cache (tables, append, varlen prefill),
    then a token each (tables, append, decode)."""
    Hq, Hkv, D, B, S, chunk = 28, 4, 128, 3, 400, 130
    m = Model(Hq, Hkv, D, False, S, 5)
    kc, vc = (torch.full((B, Hkv, S, D), float("nan"), dtype=BF16, device=DEV) for _ in range(2))
    ws = binding.decode_workspace(B, Hq, Hkv, D, S, binding.GQA_BF16, DEV)
    lens, q_lens, q_starts = i32([0] * B), ints(B), ints(B + 1)
    hist = [([], []) for _ in range(B)]
    for n, new in enumerate(([130, 7, 1], [90, 0, 128], [1, 1, 1])):
        rows = 1 if n == 2 else chunk
        T = sum(new) + (0 if n == 2 else 4)  # (a few padding tokens behind the prompts)
        pos, slots, q_slots = ints(T), ints(T), ints(T)
        binding.gqa_attn_step_tables(lens, i32(new), None, None, None, lens, q_lens, q_starts, pos, slots, q_slots,
                                     None, S, rows, ws)
        x = m.project(T, n)
        q, k, v = m.views(x)
        q_out = torch.zeros((B, Hq, rows, D), dtype=BF16, device=DEV)
        binding.gqa_attn_rope_append(q, k, v, m.wq, m.wk, m.eps, m.cs, pos, slots, q_slots, q_out, kc, vc, False, ws)
        o = torch.zeros_like(q_out)
        if n == 2:
            binding.gqa_attn_decode(q_out, kc, vc, o, lens, D ** -0.5, ws)
        else:
            binding.gqa_attn_prefill_varlen(q_out, kc, vc, o, q_lens, lens, D ** -0.5, True)
        torch.cuda.synchronize()
        positions = np.concatenate([np.arange(c) + len(hist[b][0]) for b, c in enumerate(new)] + [np.zeros(T, int)])[:T]
        kk, vv = m.keys(x, positions.astype(int))
        at = 0
        for b, c in enumerate(new):
            hist[b][0].extend(kk[at:at + c])
            hist[b][1].extend(vv[at:at + c])
            at += c
            L = len(hist[b][0])
            gk, gv = f64(kc[b, :, :L]), f64(vc[b, :, :L])
            assert ulp_close(gk, np.stack(hist[b][0], 1))
            np.testing.assert_array_equal(gv, np.stack(hist[b][1], 1))
            assert kc[b, :, L:].isnan().all()
            if c:
                ref = oracle.attention(f64(q_out[b:b + 1, :, :c]), gk[None], gv[None], scale=D ** -0.5,
                                       causal=True)["o"]
                parity.check(f64(o[b:b + 1, :, :c]), ref, "bf16", f"step {n}, request {b}")
    assert binding.gqa_attn_read_device_status(ws) == 0


def test_shared_prompt_then_own_tokens():
    """A shared prompt written once by the append, then steps in which every
    request adds tokens of its own to the same pools and attends both."""
    Hq, Hkv, D, B, bs, P = 32, 8, 128, 9, 64, 333
    m = Model(Hq, Hkv, D, False, 1000, 7)
    npb, mb = -(-P // bs), 3
    pool = npb + B * mb
    kc, vc = (torch.full((pool, Hkv, bs, D), float("nan"), dtype=BF16, device=DEV) for _ in range(2))
    ws = binding.decode_shared_prefix_workspace(B, Hq, Hkv, D, npb * bs, mb * bs)
    order = np.random.default_rng(2).permutation(pool)
    # the prompt as one request whose table is the shared rows' table
    ptable, stack, count = torch.zeros((1, npb), dtype=torch.int32, device=DEV), i32(order), i32([pool])
    plen, ql, qs = i32([0]), ints(1), ints(2)
    pos, slots = ints(P), ints(P)
    binding.gqa_attn_step_tables(plen, i32([P]), ptable, stack, count, plen, ql, qs, pos, slots, None, count, bs, P, ws)
    x = m.project(P, 0)
    q, k, v = m.views(x)
    q_prompt = torch.zeros((1, Hq, P, D), dtype=BF16, device=DEV)
    binding.gqa_attn_rope_append(q, k, v, m.wq, m.wk, m.eps, m.cs, pos, slots, None, q_prompt, kc, vc, False, ws)
    kp, vp = m.keys(x, np.arange(P))
    lens, table = i32([0] * B), torch.zeros((B, mb), dtype=torch.int32, device=DEV)
    q_lens, q_starts, pos, slots, q_slots = ints(B), ints(B + 1), ints(B), ints(B), ints(B)
    hist = [([], []) for _ in range(B)]
    for n in range(1, 71):
        binding.gqa_attn_step_tables(lens, i32([1] * B), table, stack, count, lens, q_lens, q_starts, pos, slots,
                                     q_slots, count, bs, 1, ws)
        x = m.project(B, n)
        q, k, v = m.views(x)
        q_out = torch.zeros((B, Hq, 1, D), dtype=BF16, device=DEV)
        at = pos + P  # own rows stand behind the shared ones
        binding.gqa_attn_rope_append(q, k, v, m.wq, m.wk, m.eps, m.cs, at, slots, q_slots, q_out, kc, vc, False, ws)
        o = binding.decode_shared_prefix_paged(q_out, kc, vc, ptable[0], table, lens, npb * bs, mb * bs,
                                               prefix_len=plen, workspace=ws)
        kk, vv = m.keys(x, np.full(B, P + n - 1))
        for b in range(B):
            hist[b][0].append(kk[b])
            hist[b][1].append(vv[b])
        if n in (1, 2, 63, 64, 65, 70):
            torch.cuda.synchronize()
            gkp = f64(kc[ptable[0].long()].transpose(0, 1).reshape(Hkv, npb * bs, D)[:, :P])
            gvp = f64(vc[ptable[0].long()].transpose(0, 1).reshape(Hkv, npb * bs, D)[:, :P])
            gk = f64(kc[table.long()].transpose(1, 2).reshape(B, Hkv, mb * bs, D)[:, :, :n])
            gv = f64(vc[table.long()].transpose(1, 2).reshape(B, Hkv, mb * bs, D)[:, :, :n])
            assert ulp_close(gkp, kp.transpose(1, 0, 2)) and (gvp == vp.transpose(1, 0, 2)).all()
            for b in range(B):
                assert ulp_close(gk[b], np.stack(hist[b][0], 1)) and (gv[b] == np.stack(hist[b][1], 1)).all()
            ref = oracle.attention_shared_prefix(f64(q_out), gkp, gvp, gk, gv, [n] * B, D ** -0.5)
            parity.check(f64(o), ref, "bf16", f"step {n}")
    assert binding.gqa_attn_read_device_status(ws) == 0


def test_calls_from_several_threads_and_streams():
    """The new entry points on streams of their own from several host threads
    at once give what they give one after another, bit for bit."""
    jobs = []

    def tables(seed):
        r = np.random.default_rng(seed)
        B, bs, mb = 300, 16, 20
        prior, new = i32(r.integers(0, 200, B)), i32(r.integers(-1, 30, B))
        pool = B * mb
        table0, stack0 = i32(r.integers(0, pool, (B, mb))), i32(r.permutation(pool))
        count, ws = i32([pool // 2]), torch.zeros(256, dtype=torch.uint8, device=DEV)

        def run(stream):
            with torch.cuda.stream(stream):
                t, s = table0.clone(), stack0.clone()
                outs = [ints(B), ints(B), ints(B + 1), ints(9000), ints(9000), ints(9000), ints(1)]
                binding.gqa_attn_step_tables(prior, new, t, s, count, *outs, bs, 30, ws, stream=stream)
                return [t, s, *outs]
        return run

    def append(T, seed):
        m = Model(32, 8, 128, False, 500, seed)
        x = m.project(T, 1)
        q, k, v = m.views(x)
        pos, slots = i32(np.arange(T) % 500), i32(np.random.default_rng(seed).permutation(T))
        ws = torch.zeros(256, dtype=torch.uint8, device=DEV)

        def run(stream):
            with torch.cuda.stream(stream):
                outs = [torch.zeros((T, 32, 1, 128), dtype=BF16, device=DEV),
                        *(torch.zeros((-(-T // 16), 8, 16, 128), dtype=BF16, device=DEV) for _ in range(2))]
                binding.gqa_attn_rope_append(q, k, v, m.wq, m.wk, m.eps, m.cs, pos, slots, None, *outs, False, ws,
                                             stream=stream)
                return outs
        return run

    def prefix(B, P, seed):
        q = inputs.randn((B, 28, 1, 128), seed, BF16, DEV)
        kp, vp = (inputs.randn((4, P, 128), seed + i, BF16, DEV) for i in (1, 2))
        k, v = (inputs.randn((B, 4, 100, 128), seed + i, BF16, DEV) for i in (3, 4))
        lens = i32(np.random.default_rng(seed).integers(0, 101, B))
        ws = binding.decode_shared_prefix_workspace(B, 28, 4, 128, P, 100)

        def run(stream):
            with torch.cuda.stream(stream):
                o = torch.empty_like(q)
                binding.gqa_attn_decode_shared_prefix(q, kp, vp, None, k, v, lens, o, 0.09, ws, stream=stream)
                return [o]
        return run

    jobs = [tables(1), tables(2), append(5, 3), append(3000, 4), prefix(3, 700, 500), prefix(60, 3000, 600)]
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    want = [job(s) for job, s in zip(jobs, streams)]
    torch.cuda.synchronize()
    got = [[] for _ in jobs]
    start = threading.Barrier(len(jobs))

    def work(n):
        start.wait()
        for _ in range(4):
            got[n].append(jobs[n](streams[n]))
        streams[n].synchronize()

    threads = [threading.Thread(target=work, args=(n,)) for n in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for n in range(len(jobs)):
        assert len(got[n]) == 4
        for outs in got[n]:
            assert all(torch.equal(a, b) for a, b in zip(outs, want[n])), n
