"""Drafted rows and shared pages where other tests do not look: shapes at random,
batches with long runs of idle requests, several threads and streams at once, arrays
that may not be one, and the calls that make their own workspace."""

import contextlib
import threading

import numpy as np
import pytest
import torch

import oracle
import parity
from gqa_attention_kv_decode_gb300 import binding, inputs
from test_tree_gpu import Case, f64, i32

gpu = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


@gpu
@pytest.mark.parametrize("seed", range(40))
def test_shapes_at_random(seed):
    r = np.random.default_rng(100 + seed)
    D, Hkv = int(r.choice([64, 128])), int(r.integers(1, 6))
    n_rep, B = int(r.choice([1, 2, 3, 4, 7, 8, 13])), int(r.integers(1, 7))
    Tq = int(np.exp(r.uniform(0, np.log(150))))
    N = Tq + int(r.choice([0, 0, 5, 40]))
    kv = r.integers(0, int(np.exp(r.uniform(np.log(20), np.log(2500)))) + 1, B)
    kv[0] = max(int(kv.max()), 1)
    tree = np.minimum(r.integers(0, N + 1, B), kv)
    ql = np.minimum(r.integers(0, Tq + 1, B), tree)
    chain = r.random() < 0.25
    c = Case(B, n_rep * Hkv, Hkv, D, Tq, kv, ql, None if chain else tree, N, None if chain else str(r.choice(["0.2", "0.9"])) if
             r.random() < 0.3 else "tree", S=int(kv.max()) + int(r.integers(0, 90)), seed=seed)
    c.check(int(r.choice([64, 128, 320])))


@gpu
@pytest.mark.parametrize("B,live", [(1000, [0, 1, 400, 998]), (1024, [1023]), (1025, [5, 1024]), (700, list(range(0, 700, 3)))])
@pytest.mark.parametrize("D", [64, 128])
def test_idle_requests_between_live_ones(B, live, D):
    kv, ql = np.full(B, 70), np.zeros(B, int)
    ql[live] = 3
    kv[live] = np.random.default_rng(B).integers(3, 400, len(live)) if len(live) < 10 else 71
    c = Case(B, 2, 1, D, 3, kv, ql, S=400 if len(live) < 10 else 71, mask=None)
    ref, _ = c.oracle()
    o, status = c.dense()
    assert status == 0
    parity.check(f64(o), ref, "bf16")


@gpu
def test_threads_and_streams():
    """Each thread with a stream, outputs and a workspace of its own, ten calls one after another."""
    cases = [Case(3, 16, 4, 128, 24, [900, 300, 24], seed=1), Case(5, 14, 2, 64, 4, [600, 3, 80, 200, 4], seed=2, mask=None, q_lens=[4, 3, 0, 4, 1]),
             Case(1, 8, 8, 64, 9, [2000], seed=3), Case(2, 28, 4, 128, 60, [1500, 60], seed=4)]
    got, errors = [None] * len(cases), []

    def work(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                ws = cases[i].workspace()
                for _ in range(10):
                    got[i] = cases[i].dense(ws, stream=s)[0]
            s.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for c, o in zip(cases, got):
        assert torch.equal(o, c.dense()[0])
        parity.check(f64(o), c.oracle()[0], "bf16")


@gpu
def test_a_caches_own_layers():
    """Layers of one stacked cache are what calls on each of them leave."""
    k, v = (inputs.randn((3, 9, 2, 16, 64), s, torch.bfloat16, DEV) for s in (1, 2))
    one = [(k[i].clone(), v[i].clone()) for i in range(3)]
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    path, keep, tree, lens, table = i32([[0, 3, 5], [2, 3, 9]]), i32([3, 2]), i32([8, 10]), i32([40, 33]), i32([[8, 1, 3], [0, 2, 4]])
    src, dst, rows = i32([1, -1, 4]), i32([5, 0, 6]), i32([7, 3, 16])
    out = i32([0, 0])
    binding.gqa_attn_compact_rows(path, keep, tree, lens, table, k, v, out, ws)
    binding.gqa_attn_copy_blocks(src, dst, rows, k, v, ws)
    for i, (a, b) in enumerate(one):
        binding.gqa_attn_compact_rows(path, keep, tree, lens, table, a, b, out, ws)
        binding.gqa_attn_copy_blocks(src, dst, rows, a, b, ws)
        assert torch.equal(k[i], a) and torch.equal(v[i], b)
    assert binding.gqa_attn_read_device_status(ws) == 0


@gpu
def test_arrays_that_may_not_be_one():
    k, v = (torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    a = dict(path=i32([[0, 2]]), keep=i32([2]), tree=i32([4]), lens=i32([9]), table=i32([[3]]), k=k, v=v, out=i32([7]))
    for change in (dict(out=a["lens"]), dict(out=a["keep"]), dict(out=a["tree"]), dict(v=k)):
        b = a | change
        with pytest.raises(binding.GqaAttnError) as e:
            binding.gqa_attn_compact_rows(*b.values(), ws)
        assert e.value.status == binding.GQA_ERR_INVALID_ARG
    with pytest.raises(binding.GqaAttnError) as e:
        binding.gqa_attn_copy_blocks(i32([1]), i32([2]), None, k, k, ws)
    assert e.value.status == binding.GQA_ERR_INVALID_ARG
    assert a["out"].item() == 7 and a["lens"].item() == 9


@gpu
def test_a_host_tensor_is_refused():
    k, v = (torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    calls = {
        "tree_tables": (i32([[-1, 0]]), i32([2]), i32([2]), i32([9]), i32([0, 2]), i32([[[0], [0]]]), i32([0, 0]), ws),
        "compact_rows": (i32([[0, 2]]), i32([2]), i32([4]), i32([9]), i32([[3]]), k, v, i32([7]), ws),
        "fork_tables": (i32([0]), i32([3]), i32([9]), i32([[3]]), i32([0] * 4), i32([1, 2, 0, 0]), i32([2]), i32([[0]]),
                        i32([0]), i32([0] * 4), i32([0] * 4), i32([0]), i32([0]), i32([0]), i32([0]), 16, ws),
        "copy_blocks": (i32([1]), i32([2]), i32([3]), k, v, ws),
    }
    for name, args in calls.items():
        call = getattr(binding, "gqa_attn_" + name)
        call(*args)
        for i, x in enumerate(args):
            if isinstance(x, torch.Tensor):
                with pytest.raises(binding.GqaAttnError) as e:
                    call(*args[:i], x.cpu(), *args[i + 1:])
                # (a workspace on the host may not be aligned either, which is looked at first)
                allowed = (binding.GQA_ERR_NOT_DEVICE_PTR,) + ((binding.GQA_ERR_WORKSPACE,) if x is ws else ())
                assert e.value.status in allowed, (name, i)
    torch.cuda.synchronize()


@pytest.mark.parametrize("name", ["decode_tree", "decode_tree_paged"])
@pytest.mark.parametrize("stream", [None, 77777, 0, 2])
def test_the_workspace_is_made_on_the_calls_stream(monkeypatch, name, stream):
    """(On the CPU, with stand-ins for the library's calls.)"""
    q, k = torch.zeros((2, 8, 3, 64), dtype=torch.bfloat16), torch.zeros((2, 2, 70, 64), dtype=torch.bfloat16)
    lens = torch.full((2,), 70, dtype=torch.int32)
    args = (q, k, k, lens) if name == "decode_tree" else (q, k, k, torch.zeros((2, 1), dtype=torch.int32), lens)
    on, seen = ["current"], []

    @contextlib.contextmanager
    def use(s):
        on.append(s)
        yield
        on.pop()

    monkeypatch.setattr(torch.cuda, "stream", use)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle: handle)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda: "default")
    zeros = torch.zeros
    monkeypatch.setattr(torch, "zeros", lambda *a, **kw: (seen.append(on[-1]), zeros(*a, **kw | {"device": "cpu"}))[1])
    monkeypatch.setattr(binding, "gqa_attn_" + name, lambda *a, **kw: None)
    assert getattr(binding, name)(*args, stream=stream).shape == q.shape
    assert seen == ["current" if stream is None else "default" if stream <= 2 else stream]
    seen.clear()
    getattr(binding, name)(*args, stream=stream, workspace=zeros(1 << 20, dtype=torch.uint8))
    assert seen == []


@gpu
def test_decode_is_a_tree_of_one():
    """One query without a mask is gqa_attn_decode's attention, ragged and paged."""
    lens = [700, 1, 64, 129]
    q, k, v = inputs.qkv(4, 28, 4, 128, 1, 700, torch.bfloat16, device=DEV)
    ref = oracle.attention(f64(q), f64(k), f64(v), scale=128 ** -0.5, kv_lens=np.array(lens))["o"]
    o = binding.decode_tree(q, k, v, i32(lens))
    parity.check(f64(o), ref, "bf16")
    parity.check(f64(o), f64(binding.decode(q, k, v, i32(lens))), "bf16")


@gpu
def test_a_chain_is_a_causal_chunk():
    """A chain is gqa_attn_prefill_varlen's attention of a chunk, here over pages."""
    q = inputs.randn((2, 8, 100, 64), 1, torch.bfloat16, DEV)
    k, v = (inputs.randn((2, 2, 448, 64), s, torch.bfloat16, DEV) for s in (2, 3))
    ql, kl = i32([100, 37]), i32([448, 200])
    want = torch.zeros_like(q)
    binding.gqa_attn_prefill_varlen(q, k, v, want, ql, kl, 64 ** -0.5)
    pool_k, pool_v = (x.reshape(2, 2, 7, 64, 64).transpose(1, 2).reshape(14, 2, 64, 64).contiguous() for x in (k, v))
    o = torch.zeros_like(q)
    ws = binding.decode_tree_workspace(2, 8, 2, 64, 100, 448)
    binding.gqa_attn_decode_tree_paged(q, pool_k, pool_v, i32(np.arange(14).reshape(2, 7)), None, ql, None, kl, o, 64 ** -0.5, ws)
    parity.check(f64(o), f64(want), "bf16")
