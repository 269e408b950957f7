"""gqa_attn_step_tables on the GPU: every output equal to the oracle's, and
every array it should not touch unchanged."""

import numpy as np
import pytest
import torch

import oracle
from gqa_attention_kv_decode_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda"
GUARD = -77


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def run(prior, new, T, bs, q_rows, table=None, stack=None, count=None, alias=False, q_slots=True, reps=1, stream=None):
    """The call on guarded buffers: outputs as numpy, and the status word."""
    B = len(prior)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    t = {k: dev(v) for k, v in {"prior": prior, "new": new}.items()}
    n = {"kv_lens": B, "q_lens": B, "q_starts": B + 1, "positions": T, "slots": T, "q_slots": T}
    buf = {k: torch.full((v + 64,), GUARD, dtype=torch.int32, device=DEV) for k, v in n.items()}
    out = {k: buf[k][:v] for k, v in n.items()}
    if not q_slots:
        out["q_slots"] = None
    paged = table is not None
    if paged:
        table_t, stack_t, count_t = dev(table), dev(stack), dev([count])
        out["free_count"] = count_t if alias else torch.full((1,), GUARD, dtype=torch.int32, device=DEV)
    else:
        table_t = stack_t = count_t = None
    if alias:
        out["kv_lens"], out["q_lens"] = t["prior"], t["new"]
    for _ in range(reps):
        binding.gqa_attn_step_tables(t["prior"], t["new"], table_t, stack_t, count_t, out["kv_lens"], out["q_lens"],
                                     out["q_starts"], out["positions"], out["slots"], out["q_slots"],
                                     out.get("free_count"), bs, q_rows, ws, stream=stream)
    status = binding.gqa_attn_read_device_status(ws, stream=stream)
    torch.cuda.synchronize()
    for k, v in n.items():
        if not (alias and k in ("kv_lens", "q_lens")) and not (k == "q_slots" and not q_slots):
            assert (buf[k][v:] == GUARD).all(), k
    got = {k: v.cpu().numpy() for k, v in out.items() if v is not None}
    if paged:
        got |= {"block_table": table_t.cpu().numpy(), "free_blocks": stack_t.cpu().numpy()}
        if not alias:
            assert int(count_t) == count
    return got, status


def check(*a, **kw):
    got, status = run(*a, **kw)
    prior, new, T, bs, q_rows = a[:5]
    ref = oracle.step_tables(prior, new, T, bs, q_rows, *a[5:8])
    assert status == ref.pop("status")
    for k, v in got.items():
        np.testing.assert_array_equal(v, ref[k], err_msg=k)
    return got


def draw(seed, B, bs, mb, chunk, room, release=0.1, idle=0.1, decode=0.5):
    r = np.random.default_rng(seed)
    kind = r.random(B)
    new = np.where(kind < release, -1, np.where(kind < release + idle, 0,
                   np.where(kind < release + idle + decode, 1, r.integers(1, chunk + 1, B))))
    prior = r.integers(0, mb * bs - np.maximum(new, 0) + 1)
    prior[r.random(B) < 0.2] = 0
    have = -(-prior // bs)
    pool = int(have.sum()) + max(room, 1)
    order = r.permutation(pool)
    table = np.full((B, mb), 1 << 30)  # entries of no block: never read
    at = np.concatenate([[0], np.cumsum(have)])
    for b in range(B):
        table[b, :have[b]] = order[at[b]:at[b + 1]]
    stack = np.full(pool, 1 << 30)
    stack[:room] = order[at[-1]:at[-1] + room]
    return prior, new, table, stack, room


@pytest.mark.parametrize("B", [1, 2, 31, 32, 33, 64, 300, 1023, 1024, 1025, 2500])
@pytest.mark.parametrize("bs,mb,chunk", [(64, 16, 130), (1, 40, 9), (128, 3, 300), (17, 33, 64)])
def test_random_steps(B, bs, mb, chunk):
    prior, new, table, stack, room = draw(B * 7 + bs, B, bs, mb, chunk, room=B * chunk // bs + B)
    T = int(np.maximum(new, 0).sum()) + 5
    check(prior, new, T, bs, chunk, table, stack, room)


@pytest.mark.parametrize("room", [0, 1, 7, 40, 200])
def test_too_few_blocks(room):
    prior, new, table, stack, room = draw(room + 1, 300, 16, 20, 60, room, release=0.02)
    check(prior, new, int(np.maximum(new, 0).sum()), 16, 60, table, stack, room)


@pytest.mark.parametrize("B,T", [(1, 1), (8, 3), (64, 20000), (1500, 30011), (200, 140001)])
def test_token_capacity(B, T):
    """Steps that do not fill T, or do not fit it."""
    prior, new, table, stack, room = draw(B + T, B, 64, 64, 700, room=B * 12 + B)
    check(prior, new, T, 64, 700, table, stack, room)


def test_new_blocks_of_one_long_request():
    """One request that takes hundreds of blocks in a step, one that returns as many."""
    table = np.full((3, 600), 1 << 30)
    table[1, :500] = np.arange(500)
    stack = np.full(1200, 1 << 30)
    stack[:700] = np.arange(500, 1200)
    check([0, 500 * 16 - 3, 0], [600 * 16, -1, 599 * 16 + 1], 600 * 32, 16, 600 * 16, table, stack, 700)


def test_a_decode_step_takes_a_block_only_at_a_border():
    bs = 64
    prior = np.array([0, 63, 64, 65, 127, 128, 8191, 1])
    table = np.arange(8 * 128).reshape(8, 128)
    stack = np.arange(8 * 128 + 16)[::-1].copy()
    got = check(prior, np.ones(8, int), 8, bs, 1, table, stack, 16)
    assert int(got["free_count"][0]) == 16 - 3  # rows 0, 64 and 128 begin a block


@pytest.mark.parametrize("seed", [1, 2, 3])
def test_in_place_over_many_steps(seed):
    """kv_lens over prior_lens, the count over itself: forty steps with
    requests that finish and start again, each equal to the oracle's; no block
    is ever held twice."""
    r = np.random.default_rng(seed)
    B, bs, mb, pool, chunk = 24, 16, 12, 150, 40
    prior, table = np.zeros(B, int), np.zeros((B, mb), int)
    stack, count = r.permutation(pool), pool
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    lens, table_t, stack_t, count_t = dev(prior), dev(table), dev(stack), dev([count])
    T = B * chunk
    out = {k: torch.empty(n, dtype=torch.int32, device=DEV)
           for k, n in {"q_lens": B, "q_starts": B + 1, "positions": T, "slots": T, "q_slots": T}.items()}
    for step in range(40):
        new = np.where(r.random(B) < 0.3, r.integers(0, chunk + 1, B), 1)
        new[r.random(B) < 0.08] = -1
        binding.gqa_attn_step_tables(lens, dev(new), table_t, stack_t, count_t, lens, out["q_lens"], out["q_starts"],
                                     out["positions"], out["slots"], out["q_slots"], count_t, bs, chunk, ws)
        ref = oracle.step_tables(prior, new, T, bs, chunk, table, stack, count)
        prior, table, stack, count = ref["kv_lens"], ref["block_table"], ref["free_blocks"], int(ref["free_count"][0])
        for k, v in {**out, "kv_lens": lens, "block_table": table_t, "free_blocks": stack_t,
                     "free_count": count_t}.items():
            np.testing.assert_array_equal(v.cpu().numpy(), ref[k], err_msg=f"step {step}: {k}")
        held = [int(table[b, i]) for b in range(B) for i in range(-(-int(prior[b]) // bs))] + stack[:count].tolist()
        assert sorted(held) == list(range(pool))


@pytest.mark.parametrize("alias", [False, True])
@pytest.mark.parametrize("B", [5, 1100])
def test_dense_cache(B, alias):
    r = np.random.default_rng(B)
    cap = 500
    new = np.where(r.random(B) < 0.2, -1, r.integers(0, 40, B))
    prior = r.integers(0, cap + 1, B)
    check(prior, new, int(np.maximum(new, 0).sum()) + 9, cap, 39, alias=alias)


def test_aliased_lengths_and_count():
    prior, new, table, stack, room = draw(5, 1200, 16, 20, 60, 3000)
    check(prior, new, int(np.maximum(new, 0).sum()), 16, 60, table, stack, room, alias=True)


def test_without_query_slots():
    prior, new, table, stack, room = draw(6, 20, 16, 20, 60, 300)
    check(prior, new, 400, 16, 60, table, stack, room, q_slots=False)


def test_the_same_step_again_is_the_same():
    """Nothing but the outputs changes, so a step can be run again."""
    prior, new, table, stack, room = draw(9, 100, 16, 20, 60, 900)
    check(prior, new, 3000, 16, 60, table, stack, room, reps=3)


# ------------------------------------------------ lengths and ids that are wrong

def test_out_of_range_lengths_are_clamped_and_reported():
    table = np.arange(12).reshape(4, 3)
    stack = np.arange(20)
    check([-5, 100, 4, 1 << 30], [1, 0, 2, -1], 8, 4, 2, table, stack, 8)


@pytest.mark.parametrize("big", [7, 2 ** 31 - 1])
def test_new_lens_that_fit_nothing(big):
    """Sums past 32 bits saturate; later requests get nothing, earlier ones theirs."""
    table = np.arange(12).reshape(4, 3)
    check([1, 0, 0, 2], [2, big, big, 1], 6, 4, 6, table, np.arange(20), 8)


@pytest.mark.parametrize("count", [-3, 21, 2 ** 31 - 1])
def test_a_free_count_outside_the_stack(count):
    table = np.arange(12).reshape(4, 3)
    check([0, 0, 0, 0], [4, 4, 4, 4], 16, 4, 4, table, np.arange(20), count)


@pytest.mark.parametrize("bad", [-1, 20, 2 ** 31 - 1, -2 ** 31])
def test_bad_ids_are_reported_and_their_tokens_dropped(bad):
    table = np.arange(12).reshape(4, 3)
    table[0, 0] = bad       # request 0 appends into it
    table[3, 0] = bad       # request 3 gives it back
    stack = np.arange(20)
    stack[7] = bad          # and one more is popped
    check([2, 0, 0, 5], [1, 9, 4, -1], 16, 4, 9, table, stack, 8)


def test_a_stack_with_no_room_drops_what_is_given_back():
    table = np.arange(12).reshape(4, 3)
    check([12, 12, 0, 0], [-1, -1, 1, 5], 8, 4, 5, table, np.arange(20), 17)


# ------------------------------------------------ refusals

def args(device=DEV):
    i = lambda n: torch.full((n,), 3, dtype=torch.int32, device=device)  # noqa: E731
    return dict(prior_lens=i(2), new_lens=i(2), block_table=i(8).view(2, 4), free_blocks=i(8), free_count=i(1),
                kv_lens=i(2), q_lens=i(2), q_starts=i(3), positions=i(6), slots=i(6), q_slots=i(6),
                free_count_out=i(1), block_size=16, q_rows=3,
                workspace=torch.zeros(256, dtype=torch.uint8, device=DEV))


@pytest.mark.parametrize("name", ["prior_lens", "new_lens", "block_table", "free_blocks", "free_count", "kv_lens",
                                  "q_lens", "q_starts", "positions", "slots", "q_slots", "free_count_out",
                                  "workspace"])
def test_a_host_pointer_is_refused(name):
    a = args()
    a[name] = torch.zeros_like(a[name], device="cpu")
    if name == "workspace":  # a host allocation need not be 256-byte aligned
        a[name] = torch.zeros(1024, dtype=torch.uint8).pin_memory()
    with pytest.raises(binding.GqaAttnError) as e:
        binding.gqa_attn_step_tables(**a)
    torch.cuda.synchronize()
    assert e.value.status == binding.GQA_ERR_NOT_DEVICE_PTR
    for k in ("kv_lens", "q_lens", "q_starts", "positions", "slots", "q_slots", "free_count_out"):
        assert k == name or (a[k] == 3).all()


@pytest.mark.parametrize("change,error", [
    (dict(block_size=0), binding.GQA_ERR_INVALID_ARG),
    (dict(q_rows=0), binding.GQA_ERR_INVALID_ARG),
    (dict(free_count=None), binding.GQA_ERR_INVALID_ARG),
    (dict(workspace=torch.zeros(0, dtype=torch.uint8)), binding.GQA_ERR_WORKSPACE),
])
def test_refused_arguments(change, error):
    a = args() | change
    if a["workspace"].numel() == 0:
        a["workspace"] = a["workspace"].to(DEV)
    with pytest.raises(binding.GqaAttnError) as e:
        binding.gqa_attn_step_tables(**a)
    assert e.value.status == error
    assert (a["kv_lens"] == 3).all() and (a["slots"] == 3).all()


def test_the_binding_checks_shapes_and_types():
    for change in (dict(new_lens=torch.zeros(3, dtype=torch.int32, device=DEV)),
                   dict(q_starts=torch.zeros(2, dtype=torch.int32, device=DEV)),
                   dict(slots=torch.zeros(5, dtype=torch.int32, device=DEV)),
                   dict(block_table=torch.zeros((3, 4), dtype=torch.int32, device=DEV))):
        with pytest.raises(ValueError):
            binding.gqa_attn_step_tables(**(args() | change))
    with pytest.raises(TypeError):
        binding.gqa_attn_step_tables(**(args() | dict(prior_lens=torch.zeros(2, dtype=torch.int64, device=DEV))))
