"""Shared-prefix decode on the GPU against the fp64 oracle: every request
attends the shared rows and then its own.  Bounds of a bf16 decode
(tests/parity.py).  Rows past every length are NaN unless a test says so."""

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


class Case:
    def __init__(self, B, Hq, Hkv, D, P, lens, P_cap=None, S=None, seed=0):
        self.B, self.Hq, self.Hkv, self.D, self.P = B, Hq, Hkv, D, P
        self.lens = [int(x) for x in lens]
        self.S = max(max(self.lens), 1) if S is None else S
        P_cap = max(P, 1) if P_cap is None else P_cap
        base = 900 + 10 * seed
        self.q = inputs.randn((B, Hq, 1, D), base, BF16, DEV)
        self.kp, self.vp = (inputs.randn((Hkv, P_cap, D), base + i, BF16, DEV) for i in (1, 2))
        self.k, self.v = (inputs.randn((B, Hkv, self.S, D), base + i, BF16, DEV) for i in (3, 4))
        for t in (self.kp, self.vp):
            t[:, P:] = float("nan")
        for t in (self.k, self.v):
            inputs.poison_tail(t, self.lens)
        self.scale = D ** -0.5

    def oracle(self):
        z = lambda t: np.nan_to_num(f64(t))  # noqa: E731  (NaN rows are never visible)
        return oracle.attention_shared_prefix(f64(self.q), z(self.kp)[:, :self.P], z(self.vp)[:, :self.P], z(self.k),
                                              z(self.v), self.lens, self.scale)

    def dense(self, **kw):
        return binding.decode_shared_prefix(self.q, self.kp, self.vp, self.k, self.v, prefix_len=i32([self.P]),
                                            kv_lens=i32(self.lens), **kw)

    def pools(self, bs, seed=1, spare=3):
        """Both caches scattered over one pair of pools; unused table entries
        point outside the pool."""
        npb, nb = -(-self.kp.shape[1] // bs), -(-self.S // bs)
        n = npb + self.B * nb + spare
        order = np.random.default_rng(seed).permutation(n)
        kpool = torch.full((n, self.Hkv, bs, self.D), float("nan"), dtype=BF16, device=DEV)
        vpool = torch.full_like(kpool, float("nan"))
        ptable, table = np.full(npb, 1 << 30), np.full((self.B, nb), -5)
        at = 0

        def put(k, v, rows, row_table):
            nonlocal at
            for i in range(-(-rows // bs)):
                blk, m = int(order[at]), min(bs, rows - i * bs)
                at += 1
                row_table[i] = blk
                kpool[blk, :, :m] = k[:, i * bs:i * bs + m]
                vpool[blk, :, :m] = v[:, i * bs:i * bs + m]

        put(self.kp, self.vp, self.P, ptable)
        for b in range(self.B):
            put(self.k[b], self.v[b], self.lens[b], table[b])
        return kpool, vpool, i32(ptable), i32(table)

    def paged(self, bs, max_prefix=None, max_kv=None, pools=None, **kw):
        kpool, vpool, ptable, table = self.pools(bs) if pools is None else pools
        return binding.decode_shared_prefix_paged(self.q, kpool, vpool, ptable, table, i32(self.lens),
                                                  max(self.P, 1) if max_prefix is None else max_prefix,
                                                  self.S if max_kv is None else max_kv, prefix_len=i32([self.P]), **kw)


def lens_of(B, S, seed=0):
    lens = np.random.default_rng(seed).integers(0, S + 1, B)
    lens[0] = S
    return lens


GEOMETRY = [(14, 2, 64), (28, 4, 128), (32, 8, 128), (8, 8, 64), (5, 5, 128), (24, 1, 64), (128, 1, 128), (33, 3, 64)]


@pytest.mark.parametrize("Hq,Hkv,D", GEOMETRY)
@pytest.mark.parametrize("B", [1, 3, 19, 40])
def test_geometries(Hq, Hkv, D, B):
    c = Case(B, Hq, Hkv, D, 700, lens_of(B, 90), seed=B)
    parity.check(f64(c.dense()), c.oracle(), "bf16")


@pytest.mark.parametrize("P", [1, 2, 63, 64, 65, 127, 128, 129, 255, 256, 257, 500, 1023, 1025])
@pytest.mark.parametrize("Hq,Hkv,D,B", [(14, 2, 64, 6), (32, 8, 128, 70), (28, 4, 128, 20)])
def test_prefix_lengths(P, Hq, Hkv, D, B):
    """One tile of rows and pairs of tiles, around the tile and block sizes."""
    c = Case(B, Hq, Hkv, D, P, lens_of(B, 70, P), P_cap=P + 130, seed=P)
    ref = c.oracle()
    parity.check(f64(c.dense()), ref, "bf16", "dense")
    parity.check(f64(c.paged(64)), ref, "bf16", "paged")


@pytest.mark.parametrize("bs", [64, 128, 192, 448])
@pytest.mark.parametrize("D", [64, 128])
def test_block_sizes(bs, D):
    c = Case(9, 16, 4, D, 777, lens_of(9, 500), seed=bs)
    parity.check(f64(c.paged(bs)), c.oracle(), "bf16")


@pytest.mark.parametrize("B", [31, 32, 33, 63, 64, 65, 96, 97, 130])
def test_row_tile_borders(B):
    """32 requests of four heads fill a row tile; one, two and more tiles, odd counts."""
    c = Case(B, 8, 2, 128, 400, lens_of(B, 20), seed=B)
    parity.check(f64(c.dense()), c.oracle(), "bf16")


@pytest.mark.parametrize("P,lens", [(0, [5, 1, 0, 17]), (0, [0, 0, 0, 1]), (300, [0, 0, 0, 0]), (1, [0, 1, 0, 1])])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 64), (8, 2, 128)])
def test_empty_parts(P, lens, Hq, Hkv, D):
    """No shared row, no own row, neither (a zero row and its status bit)."""
    c = Case(4, Hq, Hkv, D, P, lens, P_cap=300, S=20)
    ws = binding.decode_shared_prefix_workspace(4, Hq, Hkv, D, 300, 20)
    o = c.dense(workspace=ws)
    parity.check(f64(o), c.oracle(), "bf16")
    status = binding.gqa_attn_read_device_status(ws)
    empty = P == 0 and 0 in lens
    assert status == (binding.GQA_DEV_EMPTY_REQUEST if empty else 0)
    if empty:
        assert (o[lens.index(0)] == 0).all()
    parity.check(f64(c.paged(64, max_prefix=300)), c.oracle(), "bf16", "paged")


@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("Hq,Hkv,D", [(32, 8, 128), (14, 2, 64), (24, 1, 64), (17, 1, 128)])
def test_ragged_own_rows(Hq, Hkv, D, seed):
    """Runs of empty requests, single rows and long ones: ranges that begin and
    end anywhere in the list of tiles."""
    r = np.random.default_rng(seed)
    B = int(r.integers(1, 90))
    lens = np.where(r.random(B) < 0.3, 0, np.where(r.random(B) < 0.3, r.integers(1, 18, B), r.integers(1, 900, B)))
    lens[int(r.integers(0, B))] = 900
    c = Case(B, Hq, Hkv, D, int(r.integers(1, 300)), lens, seed=seed)
    ref = c.oracle()
    parity.check(f64(c.dense()), ref, "bf16", "dense")
    parity.check(f64(c.paged(64)), ref, "bf16", "paged")


@pytest.mark.parametrize("lens", [[5000], [4096, 3], [0, 16, 0, 5000]])
def test_long_own_rows_of_few_requests(lens):
    c = Case(len(lens), 28, 4, 128, 200, lens, seed=2)
    parity.check(f64(c.dense()), c.oracle(), "bf16")


@pytest.mark.parametrize("B", [1023, 1024, 1025, 1500])
def test_many_requests(B):
    """Up to 1,024 requests the own rows are one list, past that the decode kernel's."""
    c = Case(B, 4, 2, 64, 150, lens_of(B, 40), seed=1)
    ref = c.oracle()
    parity.check(f64(c.dense()), ref, "bf16", "dense")
    parity.check(f64(c.paged(64)), ref, "bf16", "paged")


def test_lengths_default_to_the_bounds():
    c = Case(5, 8, 2, 64, 333, [40] * 5)
    parity.check(f64(binding.decode_shared_prefix(c.q, c.kp, c.vp, c.k, c.v)), c.oracle(), "bf16")
    c = Case(5, 8, 2, 64, 200, [30] * 5, P_cap=333, S=40)
    o = binding.decode_shared_prefix(c.q, c.kp, c.vp, c.k, c.v, max_prefix_len=200, max_kv_len=30)
    parity.check(f64(o), c.oracle(), "bf16")


@pytest.mark.parametrize("P", [1, 100, 1000, 5000])
def test_capacity_sized_plans(P):
    """A plan for 8192 shared and 4096 own rows on shorter ones (graph replay)."""
    c = Case(8, 28, 4, 128, P, lens_of(8, 300), P_cap=8192, S=4096, seed=P)
    parity.check(f64(c.dense()), c.oracle(), "bf16")


@pytest.mark.parametrize("Hq,Hkv,D,B", [(32, 8, 128, 80), (14, 2, 64, 150), (40, 2, 128, 64), (16, 1, 64, 130)])
@pytest.mark.parametrize("P", [0, 129, 2500])
@pytest.mark.parametrize("own", ["none", "one", "full", "ragged", "last"])
def test_plans_that_follow_the_lengths(Hq, Hkv, D, B, P, own):
    """Grids of several SMs' worth of shares, whose number the lengths decide."""
    S = 300
    lens = {"none": [0] * B, "one": [1] * B, "full": [S] * B, "ragged": lens_of(B, S, P),
            "last": [0] * (B - 1) + [S]}[own]
    c = Case(B, Hq, Hkv, D, P, lens, P_cap=2500, S=S, seed=P + B)
    ws = binding.decode_shared_prefix_workspace(B, Hq, Hkv, D, 2500, S)
    ws[256:] = 0xFF
    parity.check(f64(c.dense(workspace=ws)), c.oracle(), "bf16")
    empty = P == 0 and min(lens) == 0
    assert binding.gqa_attn_read_device_status(ws) == (binding.GQA_DEV_EMPTY_REQUEST if empty else 0)


@pytest.mark.parametrize("S", [1, 15, 16, 17, 31, 32, 33, 47, 48, 63, 64, 65])
@pytest.mark.parametrize("D", [64, 128])
def test_own_rows_of_every_tile_remainder(S, D):
    c = Case(S + 1, 8, 2, D, 70, range(S + 1), seed=S)
    ref = c.oracle()
    parity.check(f64(c.dense()), ref, "bf16")
    parity.check(f64(c.paged(64)), ref, "bf16", "paged")


@pytest.mark.parametrize("lens", [[33, 0, 1, 32], [1055, 1056, 1057, 3], [4096, 1, 4095, 0], [1, 1, 1, 1],
                                  [2100, 31, 64, 700]])
@pytest.mark.parametrize("Hq,Hkv,D", [(14, 2, 64), (28, 4, 128), (40, 2, 128)])
def test_capacity_sized_own_rows(Hq, Hkv, D, lens):
    """Partials of a row are as many as the lengths ask for, in slots planned for 4096 own rows."""
    c = Case(4, Hq, Hkv, D, 200, lens, P_cap=8192, S=4096, seed=sum(lens))
    parity.check(f64(c.dense()), c.oracle(), "bf16")


@pytest.mark.parametrize("raw,P", [(-4, 0), (301, 300), (2 ** 31 - 1, 300), (-2 ** 31, 0)])
def test_lengths_out_of_range_are_clamped_and_reported(raw, P):
    c = Case(3, 8, 2, 64, P, [20, 7, 0], P_cap=300, S=20)
    ws = binding.decode_shared_prefix_workspace(3, 8, 2, 64, 300, 20)
    o = binding.decode_shared_prefix(c.q, c.kp, c.vp, c.k, c.v, prefix_len=i32([raw]), kv_lens=i32([21, 7, -3]),
                                     workspace=ws)
    parity.check(f64(o), c.oracle(), "bf16")
    assert binding.gqa_attn_read_device_status(ws) & binding.GQA_DEV_KVLEN_CLAMPED


def test_large_scores_need_the_running_maximum():
    """Scores that rise by hundreds along the prefix and again in the own rows."""
    c = Case(6, 8, 2, 128, 1500, [60] * 6, seed=3)
    ramp = torch.linspace(0.1, 30, 1500, device=DEV)[None, :, None]
    c.kp = (c.kp.float() * ramp).to(BF16)
    c.k[:3] = (c.k[:3].float() * 40).to(BF16)
    parity.check(f64(c.dense()), c.oracle(), "bf16")


def test_infinite_scores_of_some_keys():
    """Keys whose score is -inf for every query count nothing, wherever they
    are -- a whole share of the prefix among them."""
    c = Case(4, 8, 2, 64, 2000, [30] * 4, seed=4)
    c.q = c.q.abs() + 0.1
    c.kp[:, :1500] = float("-inf")
    want = Case(4, 8, 2, 64, 2000, [30] * 4, seed=4)
    ref = oracle.attention_shared_prefix(f64(c.q), f64(want.kp)[:, 1500:], f64(want.vp)[:, 1500:], f64(c.k), f64(c.v),
                                         c.lens, c.scale)
    parity.check(f64(c.dense()), ref, "bf16")


def test_equals_decode_over_copied_prefixes():
    """The same attention by the framework's own decode on expanded caches:
    both within their bound of the oracle, so within twice that of each other."""
    B, P, S = 12, 1000, 64
    c = Case(B, 32, 8, 128, P, [S] * B)
    k = torch.cat([c.kp[None].expand(B, -1, -1, -1), c.k], 2).contiguous()
    v = torch.cat([c.vp[None].expand(B, -1, -1, -1), c.v], 2).contiguous()
    a, b = f64(c.dense()), f64(binding.decode(c.q, k, v))
    assert np.abs(a - b).max() <= 2 * parity.REL["bf16"] * np.abs(b).max() + 1e-6


def test_long_prefix_of_a_large_batch():
    c = Case(64, 32, 8, 128, 20000, lens_of(64, 200), seed=5)
    ref = c.oracle()
    parity.check(f64(c.dense()), ref, "bf16")
    parity.check(f64(c.paged(64)), ref, "bf16")


def test_the_result_does_not_change_from_run_to_run():
    c = Case(40, 28, 4, 128, 3000, lens_of(40, 500))
    a = c.dense()
    for _ in range(3):
        assert torch.equal(a, c.dense())


def test_a_request_alone_equals_itself_in_a_batch_of_the_same_plan():
    """Rows do not mix: with NaN queries in every other request the rest stays."""
    c = Case(40, 28, 4, 128, 900, lens_of(40, 100))
    a = c.dense()
    c.q[1::2] = float("nan")
    b = c.dense()
    assert torch.equal(a[::2], b[::2]) and b[1::2].isnan().all()


def test_canaries_around_outputs_and_workspace():
    c = Case(7, 14, 2, 64, 300, lens_of(7, 50))
    n = binding.gqa_attn_decode_shared_prefix_workspace_size(7, 14, 2, 64, 300, 50)
    ws = torch.full((n + 4096,), 0xAB, dtype=torch.uint8, device=DEV)
    ws[:4] = 0
    out = torch.full((c.q.numel() + 4096,), 7.0, dtype=BF16, device=DEV)
    o = out[2048:2048 + c.q.numel()].view_as(c.q)
    binding.gqa_attn_decode_shared_prefix(c.q, c.kp, c.vp, i32([300]), c.k, c.v, i32(c.lens), o, c.scale, ws[:n])
    torch.cuda.synchronize()
    parity.check(f64(o), c.oracle(), "bf16")
    assert (ws[n:] == 0xAB).all() and (out[:2048] == 7).all() and (out[2048 + c.q.numel():] == 7).all()


def test_paged_offsets_past_32_bits():
    """Blocks beyond 2^31 elements and 2^32 bytes into the pools."""
    n, Hkv, bs, D = 4300, 8, 512, 128
    if torch.cuda.mem_get_info()[0] < 3 * n * Hkv * bs * D * 2:
        pytest.skip("not enough memory")
    c = Case(5, 32, Hkv, D, 1100, lens_of(5, 600), seed=6)
    kpool = torch.zeros((n, Hkv, bs, D), dtype=BF16, device=DEV)
    vpool = torch.zeros_like(kpool)
    small = c.pools(bs)
    off = n - small[0].shape[0]
    kpool[off:], vpool[off:] = small[0], small[1]
    o = c.paged(bs, pools=(kpool, vpool, small[2] + off, small[3] + off))
    parity.check(f64(o), c.oracle(), "bf16")


def test_bad_block_ids_are_reported_and_stay_in_the_pool():
    c = Case(4, 8, 2, 128, 400, [100] * 4)
    for which, bad in ((2, -1), (2, 1 << 20), (3, -1), (3, 1 << 20)):
        pools = list(c.pools(64))
        if which == 2:
            pools[2][2] = bad
        else:
            pools[3][1, 0] = bad
        ws = binding.decode_shared_prefix_workspace(4, 8, 2, 128, 400, 100)
        o = c.paged(64, pools=pools, workspace=ws)
        assert binding.gqa_attn_read_device_status(ws) & binding.GQA_DEV_BAD_BLOCK
        if which == 3:  # the other requests are intact
            parity.check(f64(o)[[0, 2, 3]], c.oracle()[[0, 2, 3]], "bf16")


def test_on_another_stream_and_in_a_graph():
    """Captured once, replayed with other lengths and queries in the same buffers."""
    c = Case(8, 28, 4, 128, 3000, lens_of(8, 300), P_cap=4096, S=512, seed=8)
    plen, lens = i32([c.P]), i32(c.lens)
    ws = binding.decode_shared_prefix_workspace(8, 28, 4, 128, 4096, 512)
    o = torch.empty_like(c.q)
    s = torch.cuda.Stream()

    def call(stream=None):
        binding.gqa_attn_decode_shared_prefix(c.q, c.kp, c.vp, plen, c.k, c.v, lens, o, c.scale, ws, stream=stream)

    torch.cuda.synchronize()
    call(s)
    s.synchronize()
    parity.check(f64(o), c.oracle(), "bf16", "stream")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for P, seed in ((3000, 1), (17, 2), (2048, 3)):
        other = Case(8, 28, 4, 128, P, lens_of(8, 400, seed), P_cap=4096, S=512, seed=20 + seed)
        for a, b in ((c.q, other.q), (c.kp, other.kp), (c.vp, other.vp), (c.k, other.k), (c.v, other.v)):
            a.copy_(b)
        plen.fill_(P)
        lens.copy_(i32(other.lens))
        o.zero_()
        g.replay()
        torch.cuda.synchronize()
        parity.check(f64(o), other.oracle(), "bf16", f"replay P={P}")


@pytest.mark.parametrize("Hq,Hkv,D,B", [(14, 2, 64, 4), (32, 8, 128, 4), (32, 8, 128, 80), (14, 2, 64, 80)])
@pytest.mark.parametrize("paged", [False, True])
def test_a_lost_copy_is_reported_and_the_next_call_is_right(Hq, Hkv, D, B, paged):
    """The path of a copy that never lands (see tests/test_wait_timeout_gpu.py)."""
    c = Case(B, Hq, Hkv, D, 1500, lens_of(B, 100))
    ws = binding.decode_shared_prefix_workspace(B, Hq, Hkv, D, 1500, 100)
    call = (lambda: c.paged(64, workspace=ws)) if paged else (lambda: c.dense(workspace=ws))
    call()
    torch.cuda.synchronize()
    binding.gqa_attn_set_wait_test(200_000)
    try:
        call()
        torch.cuda.synchronize()
    finally:
        binding.gqa_attn_set_wait_test(0)
    assert binding.gqa_attn_read_device_status(ws) & binding.GQA_DEV_WAIT_TIMEOUT
    binding.gqa_attn_clear_device_status(ws)
    parity.check(f64(call()), c.oracle(), "bf16")
    assert binding.gqa_attn_read_device_status(ws) == 0


@pytest.mark.parametrize("fill", [0x7F, 0xFF])
@pytest.mark.parametrize("Hq,Hkv,D,B", [(14, 2, 64, 4), (32, 8, 128, 80)])
def test_a_lost_copy_in_a_workspace_that_held_something_else(Hq, Hkv, D, B, fill):
    """The counts of partials that a lost copy leaves unwritten are not trusted."""
    c = Case(B, Hq, Hkv, D, 300, lens_of(B, 100))
    ws = binding.decode_shared_prefix_workspace(B, Hq, Hkv, D, 300, 100)
    ws[256:] = fill
    binding.gqa_attn_set_wait_test(200_000)
    try:
        c.dense(workspace=ws)
        torch.cuda.synchronize()
    finally:
        binding.gqa_attn_set_wait_test(0)
    assert binding.gqa_attn_read_device_status(ws) & binding.GQA_DEV_WAIT_TIMEOUT
    binding.gqa_attn_clear_device_status(ws)
    parity.check(f64(c.dense(workspace=ws)), c.oracle(), "bf16")
    assert binding.gqa_attn_read_device_status(ws) == 0


# ------------------------------------------------ refusals

@pytest.mark.parametrize("name", ["q", "k_prefix", "v_prefix", "prefix_len", "k", "v", "kv_lens", "o", "workspace"])
def test_a_host_pointer_is_refused(name):
    c = Case(2, 8, 2, 64, 100, [10, 20])
    a = dict(q=c.q, k_prefix=c.kp, v_prefix=c.vp, prefix_len=i32([100]), k=c.k, v=c.v, kv_lens=i32(c.lens),
             o=torch.full_like(c.q, 3.0), scale=0.125,
             workspace=binding.decode_shared_prefix_workspace(2, 8, 2, 64, 100, 20))
    o = a["o"]
    a[name] = a[name].cpu().pin_memory()
    with pytest.raises(binding.GqaAttnError) as e:
        binding.gqa_attn_decode_shared_prefix(**a)
    torch.cuda.synchronize()
    assert e.value.status == binding.GQA_ERR_NOT_DEVICE_PTR and (o == 3).all()


def test_refused_arguments():
    c = Case(2, 8, 2, 64, 100, [10, 20])
    good = dict(q=c.q, k_prefix=c.kp, v_prefix=c.vp, prefix_len=None, k=c.k, v=c.v, kv_lens=None,
                o=torch.full_like(c.q, 3.0), scale=0.125,
                workspace=binding.decode_shared_prefix_workspace(2, 8, 2, 64, 100, 20))
    for change, status in ((dict(max_prefix_len=101), binding.GQA_ERR_INVALID_ARG),
                           (dict(max_kv_len=21), binding.GQA_ERR_INVALID_ARG),
                           (dict(scale=float("nan")), binding.GQA_ERR_INVALID_ARG),
                           (dict(workspace=good["workspace"][:256]), binding.GQA_ERR_WORKSPACE),
                           (dict(workspace=good["workspace"][128:]), binding.GQA_ERR_WORKSPACE)):
        with pytest.raises(binding.GqaAttnError) as e:
            binding.gqa_attn_decode_shared_prefix(**(good | change))
        assert e.value.status == status
    f32 = {k: (v.float() if isinstance(v, torch.Tensor) and v.dtype == BF16 else v) for k, v in good.items()}
    with pytest.raises(binding.GqaAttnError) as e:
        binding.gqa_attn_decode_shared_prefix(**f32)
    assert e.value.status == binding.GQA_ERR_UNSUPPORTED
    for change in (dict(k=c.k[:1]), dict(v_prefix=c.vp[:1]), dict(k=c.k.transpose(1, 2)), dict(o=c.q[:1])):
        with pytest.raises(ValueError):
            binding.gqa_attn_decode_shared_prefix(**(good | change))
    for change in (dict(k=c.k.float()), dict(kv_lens=torch.zeros(2, dtype=torch.int64, device=DEV))):
        with pytest.raises(TypeError):
            binding.gqa_attn_decode_shared_prefix(**(good | change))
    torch.cuda.synchronize()
    assert (good["o"] == 3).all()
