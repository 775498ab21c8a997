"""The calls around the attention where offsets pass 32 bits: rows of logits, one
very long row, pages of a large cache, and more pages than a block searches."""
import pytest
import torch

import __graft_entry__
from speculative_decode_mla_tree_gb300 import abi

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    __graft_entry__.build()
    yield
    torch.cuda.empty_cache()


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def scores(x, tokens, k):
    t = x.shape[0]
    f = lambda *n: torch.full(n, 9., device="cuda")  # noqa: E731
    lp, lse, ent, ids, top = f(t), f(t), f(t), torch.full((t, k), -9, dtype=torch.int32, device="cuda"), f(t, k)
    abi.mla_token_logprobs(x, tokens, lp, lse, ent, ids, top)
    return lp, lse, ent, ids, top


def test_rows_of_logits_far_apart():
    """4 rows, 1.5e9 elements apart: each answers as a copy of it beside the others does, bit for bit."""
    v, far = 50003, 1_500_000_001
    store = torch.empty(3 * far + v, dtype=BF, device="cuda")
    x = store.as_strided((4, v), (far, 1))
    near = torch.randn(4, v, device="cuda").mul_(3).to(BF)
    x.copy_(near)
    # rows start on all kinds of addresses, as those of the copy do not: sums differ in their order
    got, want = scores(x, ints([5, 6, 7, v - 1]), 8), scores(near, ints([5, 6, 7, v - 1]), 8)
    assert torch.equal(got[3], want[3])
    lse = torch.logsumexp(near.double(), -1)
    # fp32 sums of 64 and more values a thread, then a logarithm: 2^-24 times (64 + 16) of a sum, 2^-23 of lse (about 15)
    assert float((got[1].double() - lse).abs().max()) < 80 * 2**-24 + 15 * 2**-23
    assert float((got[4] - want[4]).abs().max()) < 2 * (80 * 2**-24 + 32 * 2**-23)


@pytest.mark.parametrize("odd", [False, True], ids=["plain", "with NaN"])
def test_one_row_of_2e9_values(odd):
    """All one value but for a few: everything is known in closed form."""
    v = (1 << 31) - 3
    x = torch.full((1, v), -3., dtype=BF, device="cuda")
    marks = {0: 20., 1: 21., 2**30: 24., 2**30 + 1: 23., v - 1: 22.}
    for at, value in marks.items():
        x[0, at] = value
    if odd:
        x[0, v - 2] = float("nan")
    lp, lse, ent, ids, top = scores(x, ints([v - 1]), 7)
    order = sorted(marks, key=lambda at: -marks[at])
    rest = [at for at in range(4) if at not in marks]
    assert ids[0].tolist() == (([v - 2] if odd else []) + order + rest)[:7]
    if odd:
        assert bool(lse.isnan().all()) and bool(lp.isnan().all()) and bool(ent.isnan().all())
        return
    y = torch.tensor(list(marks.values()) + [-3.], dtype=torch.float64)
    n = torch.tensor([1.] * len(marks) + [float(v - len(marks))], dtype=torch.float64)
    want = torch.logsumexp(y + n.log(), 0)
    # a thread adds up to 2^31 / 2048 equal values in pairs: at most 2^19 roundings of 2^-24 each, of the share of e^-3 in
    # the sum (2^31 e^-27, 0.4 % of it); then a few more
    share = float(n[-1] * torch.exp(y[-1] - want))
    assert share < 0.005
    off = share * 2**19 * 2**-24 + 32 * 2**-23
    assert abs(float(lse) - float(want)) < off
    assert abs(float(lp) - (22. - float(want))) < off + 2**-18


def test_pages_of_a_large_cache():
    """Copies and compaction where rows lie beyond 2^32 elements, in pages and in layers."""
    page, pages, layers = 64, 40, 3
    stride = 150_000_000 // 8 * 8                  # 40 pages: 6e9 elements; layers inside pages
    inside = 49_999_992
    store = torch.empty(stride * (pages - 1) + inside * (layers - 1) + page * 576, dtype=BF, device="cuda")
    cache = store.as_strided((layers, pages, page, 576), (inside, stride, 576, 1))
    near = torch.randn(layers, pages, page, 576, device="cuda").to(BF)
    cache.copy_(near)
    copies = ints([[39, 0, 64], [38, 37, 13], [-1, -1, 0], [0 + 1, 36, 1]])
    abi.mla_paged_copy(copies, cache)
    near[:, 0] = near[:, 39]
    near[:, 37, :13] = near[:, 38, :13]
    near[:, 36, :1] = near[:, 1, :1]
    assert torch.equal(cache, near)
    # nodes 1, 3, 70 of a tree behind 100 positions stay
    table = ints([[35, 39, 2, 34]])
    abi.mla_paged_compact(ints([[1, 3, 70]]), ints([3]), ints([103]), table, cache)
    at = lambda pos: (slice(None), int(table[0, pos // page]), pos % page)  # noqa: E731
    for k, node in enumerate([1, 3, 70]):
        near[at(100 + k)] = near[at(100 + node)]
    assert torch.equal(cache, near)


def test_most_pages():
    """2^30 pages, all held but a few: the free ones are found, in order, by a search over 4 GB."""
    n = abi.load().mla_pages_fit_workspace_bytes(2, 1 << 30)
    refs = torch.ones(1 << 30, dtype=torch.int32, device="cuda")
    free = [7, 2**29 - 1, 2**29, 2**30 - 3, 2**30 - 1]
    refs[free] = 0
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    table, held = torch.full((2, 4), -1, dtype=torch.int32, device="cuda"), ints([0, 0])
    copies, status = torch.full((2, 3), 5, dtype=torch.int32, device="cuda"), ints([0])
    args = lambda want: (ints([0, 0]), ints(want), held, table, refs, 8, copies, ws, 0, 0, status)  # noqa: E731
    abi.mla_pages_fit(*args([32, 9]))
    assert int(status) == abi.DEV_NO_PAGES and held.tolist() == [0, 0] and int((refs == 0).sum()) == 5
    status.zero_()
    abi.mla_pages_fit(*args([24, 9]))
    assert int(status) == 0 and table[0, :3].tolist() == free[:3] and table[1, :2].tolist() == free[3:]
    assert int((refs == 1).sum()) == 1 << 30 and copies.tolist() == [[-1, -1, 0]] * 2
