"""Trees of every size in one call: what a block keeps in shared memory goes by
its own tree, what is reserved by all of them together."""
import pytest
import torch

import __graft_entry__
from speculative_decode_mla_tree_gb300 import abi

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    __graft_entry__.build()


@pytest.mark.parametrize("sizes", [[5999, 1], [6000, 0, 3], [1, 5999, 2, 400], [4095, 4096, 4097], [8192, 8191, 1, 64], [64] * 140,
                                   [1, 8192, 2048] + [9] * 300])
def test_sizes_together(sizes):
    g = torch.Generator()
    g.manual_seed(len(sizes))
    most, vocab = 40, 3
    parents, tokens, targets = [], [], []
    for n in sizes:
        parents.append([int(torch.randint(max(-1, i - 9), i, (1,), generator=g)) for i in range(n)])
        tokens.append(torch.randint(0, vocab, (n,), generator=g).tolist())
        targets.append(torch.randint(0, vocab, (n,), generator=g).tolist())
    first = torch.randint(0, vocab, (len(sizes),), generator=g).tolist()
    path, counts, ends = [], [], []
    for p, t, w, want in zip(parents, tokens, targets, first):
        children = {}
        for i in range(len(p)):
            children.setdefault((p[i], t[i]), i)
        taken, cur = [], -1
        while len(taken) < most and (cur, want) in children:
            cur = children[cur, want]
            taken.append(cur)
            want = w[cur]
        path.append(taken + [-1] * (most - len(taken)))
        counts.append(len(taken))
        ends.append(want)
    flat = lambda v: torch.tensor([x for row in v for x in row], dtype=torch.int32, device="cuda")  # noqa: E731
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    b = len(sizes)
    got = [torch.full((b, most), 7, dtype=torch.int32, device="cuda")] + [ints([7] * b) for _ in range(3)]
    lens, status = ints([n + 5 for n in sizes]), ints([0])
    indptr = torch.tensor([0] + sizes).cumsum(0).int().cuda()
    abi.mla_tree_accept(flat(parents), flat(tokens), flat(targets), indptr, lens, *got, ints(first), status)
    assert int(status) == 0 and got[0].tolist() == path and got[1].tolist() == counts and got[2].tolist() == ends
    assert got[3].tolist() == [5 + c for c in counts]
