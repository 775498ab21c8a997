"""Forks between tables that lie between one another's rows."""
import pytest
import torch

import __graft_entry__
from speculative_decode_mla_tree_gb300 import abi

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    __graft_entry__.build()


@pytest.mark.parametrize("first", [0, 1])
@pytest.mark.parametrize("old,new,width", [(1, 1, 5), (6, 6, 5), (6, 3, 1), (2, 6, 7)])
def test_interleaved_tables(old, new, width, first):
    both = torch.full((6, 2, width), -9, dtype=torch.int32, device="cuda")
    src, dst = both[:old, first], both[:new, 1 - first]
    ids = torch.arange(old * width, dtype=torch.int32, device="cuda").view(old, width)
    src.copy_(ids)
    i = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    refs = torch.ones(old * width, dtype=torch.int32, device="cuda")
    held, lens = i(*[width] * old), i(*range(old))
    parents = [(3 * r + 1) % old for r in range(new)]
    nh, nl, status = i(*[0] * new), i(*[0] * new), i(0)
    abi.mla_pages_fork(i(*parents), lens, held, src, refs, nl, nh, dst, status)
    assert int(status) == 0 and torch.equal(dst, ids[parents]) and torch.equal(src, ids)
    assert nl.tolist() == parents and nh.tolist() == [width] * new
    assert refs.view(old, width).tolist() == [[parents.count(s)] * width for s in range(old)]
    assert (both[new:, 1 - first] == -9).all() and (both[old:, first] == -9).all()
