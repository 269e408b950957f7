"""Arrays of the forked tables and the tree tables that may be one, and those that may not
(refused on the host; the pointers are never read)."""

import ctypes

import pytest

from gqa_attention_kv_decode_gb300 import binding
from test_tree_pages import AT, INVALID, REACHES_THE_DEVICE, fork, lib  # noqa: F401  (lib: a fixture)

IN_PLACE = {"shared_out": "shared", "stack_out": "stack", "count_out": "count"}


@pytest.mark.parametrize("now", list(IN_PLACE))
@pytest.mark.parametrize("before", list(IN_PLACE.values()))
def test_holders_stack_and_count_may_be_their_own_inputs_only(lib, now, before):  # noqa: F811
    got = fork(lib, **{now: AT[before]})
    assert got in REACHES_THE_DEVICE if IN_PLACE[now] == before else got == INVALID


def test_all_three_in_place(lib):  # noqa: F811
    assert fork(lib, **{now: AT[before] for now, before in IN_PLACE.items()}) in REACHES_THE_DEVICE


def tables(lib, **change):  # noqa: F811
    a = {x: ctypes.c_void_p(256 * (i + 2)) for i, x in enumerate(("parents", "n", "q", "kv", "starts", "mask", "pos"))} | change
    return lib.gqa_attn_tree_tables(*(a[x] for x in ("parents", "n", "q", "kv", "starts", "mask", "pos")), 2, 40, 8, 2, 16,
                                    AT["src"], 256, None)


@pytest.mark.parametrize("now", ["mask", "pos"])
@pytest.mark.parametrize("before", ["parents", "n", "q", "kv", "starts", "mask"])
def test_masks_and_positions_are_arrays_of_their_own(lib, now, before):  # noqa: F811
    """A block writes them while another one reads its parents and lengths."""
    if now != before:
        at = dict(zip(("parents", "n", "q", "kv", "starts", "mask"), (ctypes.c_void_p(256 * (i + 2)) for i in range(6))))
        assert tables(lib, **{now: at[before]}) == INVALID


def test_tree_tables_without_positions_or_query_lengths(lib):  # noqa: F811
    assert tables(lib) in REACHES_THE_DEVICE
    assert tables(lib, q=None) in REACHES_THE_DEVICE
    assert tables(lib, kv=None, starts=None, pos=None) in REACHES_THE_DEVICE
    assert tables(lib, q=None, kv=None, starts=None, pos=None) in REACHES_THE_DEVICE
