"""Own rows of a shared-prefix decode near 2^31, whose tiles and splits would
not fit 32 bits, are refused before anything reaches the device (CPU)."""

import ctypes

import pytest

import __graft_entry__
from gqa_attention_kv_decode_gb300 import binding

P = ctypes.c_void_p(256)  # never dereferenced: shape checks come first
MOST = 1 << 30


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    return binding.lib()


@pytest.mark.parametrize("L", [MOST + 1, 2 ** 31 - 256, 2 ** 31 - 32, 2 ** 31 - 1])
@pytest.mark.parametrize("B", [1, 2000])
def test_longer_own_rows_are_refused(lib, B, L):
    assert binding.gqa_attn_decode_shared_prefix_workspace_size(B, 1, 1, 64, 100, L) == 0
    assert lib.gqa_attn_decode_shared_prefix(P, P, P, P, P, P, P, P, B, 1, 1, 64, 100, 100, L, L, 0.1, 1, P, 1 << 40,
                                             None) == binding.GQA_ERR_INVALID_ARG
    assert lib.gqa_attn_decode_shared_prefix_paged(P, P, P, P, P, P, P, P, B, 1, 1, 64, 64, 20, 2, 1 << 25, 100, L,
                                                   0.1, 1, P, 1 << 40, None) == binding.GQA_ERR_INVALID_ARG


@pytest.mark.parametrize("B", [1, 64, 1025, 65535])
@pytest.mark.parametrize("variant", [binding.GQA_PLAN_DECODE, binding.GQA_PLAN_PAGED])
def test_the_longest_ones_fit_32_bits(lib, B, variant):
    """The sums the kernels make of a length: rounded up to tiles of 32 and 128
    keys, and to a split of the decode kernel's plan."""
    assert binding.gqa_attn_decode_shared_prefix_workspace_size(B, 1, 1, 64, 100, MOST) > 0
    n_split, chunk, tile = binding.gqa_attn_decode_plan_for(B, 1, 1, 64, MOST, binding.GQA_BF16, 152, variant)
    assert max(MOST + 31, MOST + 127, MOST + chunk - 1, n_split * chunk + chunk, MOST + tile - 1) < 2 ** 31
