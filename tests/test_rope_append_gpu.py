"""gqa_attn_rope_append on the GPU against the fp64 oracle.

Bounds, from the arithmetic (u = 2^-24, the fp32 rounding; D = 128 at most).
A normed value x * inv * w: the mean of squares is a sum of D products in some
order, off by at most (D + 1) u of itself, half of that in its root; rsqrtf is
within 2 ulp (2^-22 = 4 u); two products round once each: together
(D / 2 + 8) u, 72 u at D = 128.  The rotated value a c - b s is a product and
a fused or separate product and difference: 3 u (|a c| + |b s|), on top of
what a and b bring.  So fp32 outputs lie within 76 u (|a c| + |b s|), a bf16
output within half a bf16 step (2^-9 of the value's binade, at most 2^-8 of
the value) more.  Values that are neither normed nor rotated, and V, are
copies.
"""

import numpy as np
import pytest
import torch

import oracle
from gqa_attention_kv_decode_gb300 import binding, inputs

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def f64(t):
    return t.detach().double().cpu().numpy()


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


class Case:
    """Inputs of a call: a projection output whose q, k, v are views, caches
    and query buffer filled with values that must survive."""

    def __init__(self, T, Hq, Hkv, D, dtype, rot=None, adjacent=False, norm="qk", bs=16, q_rows=1, seed=0,
                 max_pos=5000, pad=0, gap=0, identity_q=False):
        r = np.random.default_rng(seed)
        rot = D if rot is None else rot
        self.adjacent, self.eps, self.T, self.D = adjacent, 1e-5, T, D
        width = (Hq + 2 * Hkv) * D + gap
        base = 50 * seed + 3
        x = inputs.randn((T, width), base, dtype, DEV)
        self.q, self.k, self.v = (y.unflatten(1, (-1, D)) for y in
                                  x[:, :(Hq + 2 * Hkv) * D].split([Hq * D, Hkv * D, Hkv * D], dim=1))
        self.wq = inputs.randn((D,), base + 1, dtype, DEV) if "q" in norm else None
        self.wk = inputs.randn((D,), base + 2, dtype, DEV) if "k" in norm else None
        self.cs = binding.rope_table(max_pos, rot) if rot else None
        self.pos = i32(r.integers(0, max_pos, T)) if rot else None
        nb = -(-T // bs) + 3
        slots = r.permutation(nb * bs)[:T]
        groups = -(-T // q_rows) + 1
        q_slots = r.permutation(groups * q_rows)[:T]
        if pad:
            lost = r.permutation(T)
            slots[lost[:pad]] = -1
            q_slots[lost[pad // 2:pad // 2 + pad]] = -5
        self.slots, self.q_slots = i32(slots), None if identity_q else i32(q_slots)
        self.q_out = inputs.randn((groups, Hq, q_rows, D), base + 4, dtype, DEV)
        self.kc = inputs.randn((nb, Hkv, bs, D), base + 5, dtype, DEV)
        self.vc = inputs.randn((nb, Hkv, bs, D), base + 6, dtype, DEV)

    def call(self, ws, stream=None, **over):
        a = {"q": self.q, "k": self.k, "v": self.v, "q_weight": self.wq, "k_weight": self.wk, "eps": self.eps,
             "cos_sin": self.cs, "positions": self.pos, "slots": self.slots, "q_slots": self.q_slots,
             "q_out": self.q_out, "k_cache": self.kc, "v_cache": self.vc, "adjacent": self.adjacent} | over
        binding.gqa_attn_rope_append(*a.values(), ws, stream=stream)

    def oracle(self):
        num = lambda t: None if t is None else t.cpu().numpy()  # noqa: E731
        w = lambda t: None if t is None else f64(t)  # noqa: E731
        return oracle.rope_append(f64(self.q), f64(self.k), f64(self.v), w(self.wq), w(self.wk), self.eps, w(self.cs),
                                  num(self.pos), num(self.slots), num(self.q_slots), f64(self.q_out), f64(self.kc),
                                  f64(self.vc), self.adjacent)

    def spread(self):
        """|a c| + |b s| of every output element: the oracle with |.| of every term."""
        num = lambda t: None if t is None else t.cpu().numpy()  # noqa: E731
        w = lambda t: None if t is None else np.abs(f64(t))  # noqa: E731
        cs = None
        if self.cs is not None:  # |cos| for the first term, -|sin| and |sin|: both terms add up
            cs = np.abs(f64(self.cs))
        q, k = np.abs(f64(self.q)), np.abs(f64(self.k))
        out = []
        for x, wt in ((q, w(self.wq)), (k, w(self.wk))):
            y = oracle.rms_norm(x, wt, self.eps)
            if cs is not None:
                p = num(self.pos) % cs.shape[0]
                R = cs.shape[1]
                a = oracle.rotate(y, cs[p][:, :R // 2], np.zeros((self.T, R // 2)), self.adjacent)
                b = oracle.rotate(y, np.zeros((self.T, R // 2)), cs[p][:, R // 2:], self.adjacent)
                y = np.abs(a) + np.abs(b)
                y[..., R:] = np.abs(a[..., R:])
            out.append(y)
        return out


def check(c, ws=None, **kw):
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV) if ws is None else ws
    before = [t.clone() for t in (c.q_out, c.kc, c.vc)]
    qo, kc, vc, status = c.oracle()
    sq, sk = c.spread()
    c.call(ws, **kw)
    assert binding.gqa_attn_read_device_status(ws) == status
    torch.cuda.synchronize()
    # V and untouched rows: bit for bit
    np.testing.assert_array_equal(f64(c.vc), vc)
    half_step = 2.0 ** -8 if c.q.dtype == torch.bfloat16 else U
    q_slots = np.arange(c.T) if c.q_slots is None else c.q_slots.cpu().numpy()
    for got, ref, spread, slots, old, wt in ((c.q_out, qo, sq, q_slots, before[0], c.wq),
                                             (c.kc, kc, sk, c.slots.cpu().numpy(), before[1], c.wk)):
        rows, H = got.shape[2], got.shape[1]
        touched = np.zeros((got.shape[0], rows), dtype=bool)
        bound = np.zeros(ref.shape)
        for t in range(c.T):
            if 0 <= slots[t] < got.shape[0] * rows:
                g, r = divmod(int(slots[t]), rows)
                touched[g, r] = True
                bound[g, :, r] = 76 * U * spread[t] + half_step * np.abs(ref[g, :, r])
                R = 0 if c.cs is None else c.cs.shape[1]
                if wt is None:  # neither normed nor rotated: copies
                    bound[g, :, r, R:] = 0.0
        assert (np.abs(f64(got) - ref) <= bound).all()
        keep = ~torch.from_numpy(touched).to(DEV)[:, None, :, None].expand_as(got)
        assert torch.equal(got[keep], old[keep])


GEOMETRY = [(14, 2, 64), (28, 4, 128), (32, 8, 128), (1, 1, 64), (5, 5, 128), (16, 1, 64), (9, 3, 128)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hkv,D", GEOMETRY)
@pytest.mark.parametrize("T", [1, 7, 65])
def test_geometries(dtype, Hq, Hkv, D, T):
    check(Case(T, Hq, Hkv, D, dtype, seed=T))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("adjacent", [False, True], ids=["half", "adjacent"])
@pytest.mark.parametrize("D,rot", [(64, 0), (64, 16), (64, 32), (64, 48), (64, 64), (128, 16), (128, 80), (128, 112),
                                   (128, 128)])
@pytest.mark.parametrize("norm", ["qk", "q", "k", ""], ids=["qk", "q", "k", "none"])
def test_rotations_and_norms(dtype, adjacent, D, rot, norm):
    check(Case(9, 6, 2, D, dtype, rot=rot, adjacent=adjacent, norm=norm, seed=rot + D))


@pytest.mark.parametrize("T", [1000, 4097])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_many_tokens(T, dtype):
    check(Case(T, 14, 2, 64, dtype, q_rows=37, bs=64, seed=T, pad=T // 5))


def test_many_tokens_of_wide_heads():
    check(Case(2001, 32, 8, 128, torch.bfloat16, q_rows=512, bs=64, seed=4, pad=17))


@pytest.mark.parametrize("dtype,Hq,Hkv,D,T", [(torch.bfloat16, 32, 8, 128, 1500), (torch.bfloat16, 14, 2, 64, 4001),
                                              (torch.float32, 28, 4, 128, 1300), (torch.float32, 9, 3, 64, 3000),
                                              (torch.bfloat16, 7, 7, 64, 4000), (torch.bfloat16, 16, 1, 128, 2500),
                                              (torch.float32, 64, 16, 128, 600), (torch.bfloat16, 96, 96, 128, 200)])
@pytest.mark.parametrize("kind", ["half", "adjacent", "part", "plain", "one-norm"])
def test_many_tokens_of_every_kind(dtype, Hq, Hkv, D, T, kind):
    """Steps of several waves of blocks, and, at the smallest head counts, of one
    pass of heads a warp."""
    kw = {"half": {}, "adjacent": dict(adjacent=True), "part": dict(rot=48, pad=T // 3, gap=64, q_rows=100),
          "plain": dict(rot=0, norm="", identity_q=True), "one-norm": dict(norm="k", rot=D - 16, adjacent=True)}[kind]
    check(Case(T, Hq, Hkv, D, dtype, bs=64, seed=20, **kw))


@pytest.mark.parametrize("dtype,T", [(torch.bfloat16, 5501), (torch.float32, 2751)], ids=["bf16", "f32"])
def test_outputs_of_more_than_half_of_l2(dtype, T):
    check(Case(T, 32, 8, 128, dtype, q_rows=512, bs=64, seed=24, pad=99, gap=64))


def test_many_tokens_with_bad_places():
    c = Case(3000, 14, 2, 64, torch.bfloat16, bs=64, seed=21, pad=100)
    c.pos[5], c.pos[2999], c.slots[700], c.q_slots[701] = -1, 5000, 2 ** 31 - 1, c.q_out.shape[0] * c.q_out.shape[2]
    check(c)


def test_many_padding_tokens():
    """Runs of padding that leave whole blocks with nothing to do."""
    c = Case(40000, 2, 2, 64, torch.bfloat16, bs=64, seed=22)
    c.slots[100:39000] = -1
    c.q_slots[90:39500] = -1
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    qo, kc, vc, _ = c.oracle()
    c.call(ws)
    np.testing.assert_array_equal(f64(c.vc), vc)
    assert np.abs(f64(c.q_out) - qo).max() <= 2.0 ** -8 * np.abs(qo).max() + 76 * U * 20


@pytest.mark.parametrize("gap", [8, 64])
def test_token_strides(gap):
    check(Case(33, 14, 2, 64, torch.bfloat16, gap=gap, seed=5))


def test_separate_tensors_and_row_order():
    c = Case(12, 8, 4, 64, torch.bfloat16, q_rows=4, seed=6, identity_q=True)
    c.q, c.k, c.v = c.q.contiguous(), c.k.contiguous(), c.v.contiguous()
    check(c)


def test_dense_cache_is_a_pool_of_one_block_a_request():
    """Slot b * S_cap + row writes row `row` of request b of a [B,Hkv,S_cap,D] cache."""
    c = Case(3, 8, 4, 64, torch.bfloat16, bs=50, seed=7, norm="", rot=0)
    c.slots = i32([0 * 50 + 7, 2 * 50 + 49, 1 * 50 + 0])
    check(c)
    for t, (b, r) in enumerate(((0, 7), (2, 49), (1, 0))):
        assert torch.equal(c.kc[b, :, r], c.k[t]) and torch.equal(c.vc[b, :, r], c.v[t])


@pytest.mark.parametrize("T,pad", [(8, 8), (40, 10)])
def test_padding_tokens_write_nothing(T, pad):
    check(Case(T, 6, 2, 128, torch.bfloat16, pad=pad, seed=8))


def test_padding_positions_are_not_looked_at():
    c = Case(6, 6, 2, 64, torch.bfloat16, seed=9)
    c.slots[2], c.q_slots[2], c.pos[2] = -1, -1, 10 ** 6
    check(c)


@pytest.mark.parametrize("pos", [-1, 5000, 2 ** 31 - 1, -2 ** 31])
def test_bad_positions_are_reported_and_skipped(pos):
    c = Case(6, 6, 2, 64, torch.bfloat16, seed=10)
    c.pos[4] = pos
    check(c)


@pytest.mark.parametrize("slot", ["past", 2 ** 31 - 1])
@pytest.mark.parametrize("which", ["slots", "q_slots"])
def test_bad_slots_are_reported_and_skipped(slot, which):
    c = Case(6, 6, 2, 64, torch.bfloat16, seed=11)
    n = c.kc.shape[0] * c.kc.shape[2] if which == "slots" else c.q_out.shape[0] * c.q_out.shape[2]
    getattr(c, which)[3] = n if slot == "past" else slot
    check(c)


def test_zero_rows_and_infinities():
    """A zero head row norms to zeros (eps keeps the root finite); infinities
    and NaN stay in the head they came in, and V carries them unchanged."""
    c = Case(4, 4, 2, 64, torch.float32, seed=12, rot=0)
    c.q[0, 1] = 0.0
    c.v[1, 0, 5] = float("inf")
    c.v[1, 1, 6] = float("nan")
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    c.call(ws)
    g, r = divmod(int(c.q_slots[0]), c.q_out.shape[2])
    assert (c.q_out[g, 1, r] == 0).all()
    g, r = divmod(int(c.slots[1]), c.kc.shape[2])
    assert torch.equal(c.vc[g, :, r].view(torch.int32), c.v[1].view(torch.int32))
    c.k[2, 0, 3] = float("nan")
    c.call(ws)
    g, r = divmod(int(c.slots[2]), c.kc.shape[2])
    assert c.kc[g, 0, r].isnan().all() and c.kc[g, 1, r].isfinite().all()


def test_offsets_past_32_bits():
    """A pool of more than 2^32 bytes and 2^31 elements: the last rows."""
    nb, Hkv, bs, D = 4200, 64, 64, 128
    if torch.cuda.mem_get_info()[0] < 3 * nb * Hkv * bs * D * 2:
        pytest.skip("not enough memory")
    c = Case(3, 64, 64, 128, torch.bfloat16, seed=13)
    kc = torch.zeros((nb, Hkv, bs, D), dtype=torch.bfloat16, device=DEV)
    vc = torch.zeros_like(kc)
    c.slots = i32([nb * bs - 1, 5, (nb - 1) * bs])
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    c.call(ws, k_cache=kc, v_cache=vc)
    assert torch.equal(vc[nb - 1, :, bs - 1], c.v[0]) and torch.equal(vc[0, :, 5], c.v[1])
    assert torch.equal(vc[nb - 1, :, 0], c.v[2])
    assert int((vc != 0).any(-1).sum()) == 3 * Hkv and int((kc != 0).any(-1).sum()) == 3 * Hkv
    assert binding.gqa_attn_read_device_status(ws) == 0


def test_on_another_stream():
    s = torch.cuda.Stream()
    c = Case(500, 32, 8, 128, torch.bfloat16, seed=14)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    ref = c.oracle()
    c.call(ws, stream=s)
    s.synchronize()
    np.testing.assert_array_equal(f64(c.vc), ref[2])


# ------------------------------------------------ refusals

@pytest.mark.parametrize("name", ["q", "k", "v", "q_weight", "k_weight", "cos_sin", "positions", "slots", "q_slots",
                                  "q_out", "k_cache", "v_cache"])
def test_a_host_pointer_is_refused(name):
    c = Case(5, 4, 2, 64, torch.bfloat16, seed=15)
    old = [t.clone() for t in (c.q_out, c.kc, c.vc)]
    field = {"q_weight": c.wq, "k_weight": c.wk, "cos_sin": c.cs, "positions": c.pos, "k_cache": c.kc,
             "v_cache": c.vc}.get(name)
    field = getattr(c, name) if field is None else field
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    with pytest.raises(binding.GqaAttnError) as e:
        c.call(ws, **{name: field.cpu().contiguous().pin_memory()})
    torch.cuda.synchronize()
    assert e.value.status == binding.GQA_ERR_NOT_DEVICE_PTR
    assert all(torch.equal(a, b) for a, b in zip(old, (c.q_out, c.kc, c.vc)))


def test_the_binding_checks_shapes_types_and_strides():
    c = Case(5, 4, 2, 64, torch.bfloat16, seed=16)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    wide = torch.zeros((5, 2, 128), dtype=torch.bfloat16, device=DEV)
    for bad in (dict(k=c.k[:4]), dict(v=c.v[:, :1]), dict(q_out=c.q_out[:, :2]), dict(v_cache=c.vc[:1]),
                dict(q_weight=c.wq[:32]), dict(slots=c.slots[:4]), dict(q_slots=c.q_slots[:2]),
                dict(k=wide[:, :, ::2]), dict(q=torch.zeros((5, 8, 64), dtype=torch.bfloat16, device=DEV)[:, ::2])):
        with pytest.raises(ValueError):
            c.call(ws, **bad)
    for bad in (dict(k=c.k.float()), dict(q_weight=c.wq.float()), dict(v_cache=c.vc.float()),
                dict(cos_sin=c.cs.double()), dict(positions=None), dict(slots=c.slots.long())):
        with pytest.raises(TypeError):
            c.call(ws, **bad)
    with pytest.raises(binding.GqaAttnError) as e:  # a row that does not start on 16 bytes
        c.call(ws, q=torch.zeros((5, 4 * 64 + 4), dtype=torch.bfloat16, device=DEV)[:, :256].unflatten(1, (4, 64)))
    assert e.value.status == binding.GQA_ERR_INVALID_ARG
    with pytest.raises(binding.GqaAttnError) as e:
        c.call(torch.zeros(0, dtype=torch.uint8, device=DEV))
    assert e.value.status == binding.GQA_ERR_WORKSPACE
