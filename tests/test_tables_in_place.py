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
