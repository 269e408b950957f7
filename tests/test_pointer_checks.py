"""The lookup of pointers (gqa_attn_set_pointer_checks): on unless a thread turns
it off for itself, and never all there is between a call and a bad argument."""

import threading

import pytest
import torch

import __graft_entry__
from gqa_attention_kv_decode_gb300 import binding


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    return binding.lib()


def test_it_is_on_and_returns_the_setting_before(lib):
    assert lib.gqa_attn_set_pointer_checks(0) == 1
    assert lib.gqa_attn_set_pointer_checks(0) == 0
    assert lib.gqa_attn_set_pointer_checks(1) == 0
    assert binding.gqa_attn_set_pointer_checks(True) is True
    for on in (-1, 2, 7):
        assert lib.gqa_attn_set_pointer_checks(on) == binding.GQA_ERR_INVALID_ARG
    assert lib.gqa_attn_set_pointer_checks(1) == 1


def test_it_is_a_threads_own(lib):
    seen = []
    lib.gqa_attn_set_pointer_checks(0)
    try:
        t = threading.Thread(target=lambda: seen.append(lib.gqa_attn_set_pointer_checks(1)))
        t.start()
        t.join()
    finally:
        assert lib.gqa_attn_set_pointer_checks(1) == 0
    assert seen == [1]


@pytest.mark.parametrize("q", [None, 257])
def test_null_and_misaligned_pointers_are_refused_without_it(lib, q):
    """(Without a device the call ends before it comes to the pointers.)"""
    lib.gqa_attn_set_pointer_checks(0)
    try:
        rc = lib.gqa_attn_decode_shared_prefix(q, 256, 256, None, 256, 256, None, 256, 1, 2, 2, 64, 128, 128, 128, 128,
                                               0.125, binding.GQA_BF16, 256, 1 << 20, None)
    finally:
        lib.gqa_attn_set_pointer_checks(1)
    assert rc in (binding.GQA_ERR_INVALID_ARG, binding.GQA_ERR_CUDA)


@pytest.mark.gpu
def test_a_host_tensor_among_the_others_is_looked_up(lib):
    """The tensors say where they are; one on the host leaves the lookups on."""
    n = {k: torch.zeros(2, dtype=torch.int32, device="cuda") for k in "abcdefg"}
    starts, ws = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.zeros(256, dtype=torch.uint8, device="cuda")
    args = [n["a"], n["b"], None, None, None, n["c"], n["d"], starts, n["e"], n["f"], n["g"], None, 8, 1, ws]
    binding.gqa_attn_step_tables(*args)
    for i in (0, 1, 5, 6, 7, 8, 9, 10, 14):
        bad = list(args)
        bad[i] = args[i].cpu()
        with pytest.raises(binding.GqaAttnError):
            binding.gqa_attn_step_tables(*bad)
    assert lib.gqa_attn_set_pointer_checks(1) == 1
    torch.cuda.synchronize()
