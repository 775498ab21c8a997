"""Forks between tables that share memory in part are refused before anything is
launched, however their rows lie."""
import pytest

import __graft_entry__
from speculative_decode_mla_tree_gb300 import abi

from test_around_cpu import FAKE, call

BASE = 16 * FAKE


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build_library()
    return abi.load()


@pytest.mark.parametrize("at,new_stride,new", [
    (0, 10, 6),       # the same rows
    (4, 10, 6),       # one number of each
    (-4, 10, 1),
    (5, 9, 6),        # between one another at first
    (5, 11, 6),
    (54, 10, 1),      # the last row's last number
    (-54, 10, 6),
    (-36, 9, 6),
])
def test_tables_that_share_a_number(lib, at, new_stride, new):
    """Six rows of 5 numbers, 10 apart, and others."""
    assert call(lib, "mla_pages_fork", table=BASE, table_stride=10, old=6, max_pages=5, new_table=BASE + 4 * at,
                new_stride=new_stride, new=new) == abi.MT_EINVAL
