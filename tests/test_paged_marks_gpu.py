"""Every key counts once: decode on marked keys, wherever tiles, shares and pages
end, and on drawn ones by the usual size of the error."""

import pytest
import torch

import __graft_entry__

import paged_marks as marks
import paged_ref as ref
from test_paged_gpu import BF, SCALE, decode, gen, normal, paged

pytestmark = pytest.mark.gpu

LAYOUTS = pytest.mark.parametrize("page,gap", [(64, 0), (16, 0), (24, 0), (1, 0), (20, 8)])
BATCHES = {"long": [20011], "longest": [50000], "odd": [12000, 1, 9001, 0, 3, 64, 65], "short": [1, 63, 64, 65, 127, 129] * 40,
           "many": [500] * 160, "few tiles": [640, 577, 1000, 321] * 5, "uneven": [30000, 2, 100, 8192, 0, 40000]}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    __graft_entry__.build()


def run(seed, lens, heads, page, gap, q=None, values=None):
    g = gen(seed)
    cache, flat, table = paged(g, lens, page, gap=gap)
    if values:
        for b, n in enumerate(lens):
            flat[ref.slots_of(table[b], page, 0, n), :512] = values[b].to(BF)
        cache.copy_(flat.view(cache.shape))
    q = torch.zeros(len(lens), heads, 576, dtype=BF) if q is None else q
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = decode(q.cuda(), cache, table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), status)
    assert int(status) == 0
    return out.cpu(), lse.cpu(), flat, table


@LAYOUTS
@pytest.mark.parametrize("batch", sorted(BATCHES))
@pytest.mark.parametrize("heads", [8, 64])
def test_decode_counts_every_key_once(heads, batch, page, gap):
    lens, g = BATCHES[batch], gen(90)
    kinds = {n: marks.marked(g, n) for n in set(lens)}
    out, lse, _, _ = run(91, lens, heads, page, gap, values=[kinds[n][0] for n in lens])
    for b, n in enumerate(lens):
        if n:
            marks.check_marks(out[b], lse[b], n, kinds[n][1])
        else:
            assert (out[b] == 0).all() and torch.isneginf(lse[b]).all()


@pytest.mark.parametrize("heads", [24, 65, 128, 200])
@pytest.mark.parametrize("page", [32, 3])
def test_decode_counts_every_key_once_more_heads(heads, page):
    lens, g = [7000, 0, 129, 20011, 64], gen(92)
    kinds = [marks.marked(g, n) for n in lens]
    out, lse, _, _ = run(93, lens, heads, page, 0, values=[v for v, _ in kinds])
    for b in (0, 2, 3, 4):
        marks.check_marks(out[b], lse[b], lens[b], kinds[b][1])


@pytest.mark.parametrize("n", list(range(180, 260)))
def test_decode_counts_every_key_once_at_every_tail(n):
    """All remainders of a tile and of a page, in one request and a batch of two."""
    g = gen(n)
    values, counts = marks.marked(g, n)
    for page in (64, 24, 7):
        out, lse, _, _ = run(n, [n, n], 16, page, 0, values=[values, values])
        for b in range(2):
            marks.check_marks(out[b], lse[b], n, counts)


@pytest.mark.parametrize("page,gap", [(64, 0), (24, 0), (1, 0), (20, 8)])
@pytest.mark.parametrize("lens,heads", [([20011], 8), ([20011], 64), ([3000, 1000, 12000], 24), ([1500] * 20, 64),
                                        ([5000, 2000], 128)], ids=["20011-8", "20011-64", "ragged", "batch", "128"])
def test_decode_drawn_by_the_usual_error(lens, heads, page, gap):
    q = normal(gen(94), len(lens), heads, 576) / 2
    out, lse, flat, table = run(95, lens, heads, page, gap, q)
    want = ref.decode(q, flat, table, lens, page, SCALE)
    marks.check_close(out, lse, want[0], want[1])
