"""What follows a call that found too few pages: nothing may be written, and a
program that does not look at the status between its calls has to be told by
what the next ones read."""
import math

import pytest
import torch

import __graft_entry__
from speculative_decode_mla_tree_gb300 import abi
from speculative_decode_mla_tree_gb300.step import DecodeStep, Pages

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
SCALE = 1.0 / math.sqrt(192.0)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    __graft_entry__.build()


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("captured", [False, True])
def test_branches_without_pages_write_nothing(captured):
    """Two branches share their last page and the pool has none left: neither may write to it."""
    pages = Pages(1, 2, 4, 2, 3)
    rope = torch.cat([torch.ones(16, 32), torch.zeros(16, 32)], 1).cuda()
    step = DecodeStep(pages.cache[0], 2, 8, 3, rope, SCALE)
    pages.want_lens[0] = 6
    pages.fit()
    pages.cache.copy_(torch.arange(8, dtype=BF, device="cuda").view(1, 2, 4, 1).expand_as(pages.cache))
    pages.advance()
    assert pages.kv_lens.tolist() == [6, 0] and pages.step_lens.tolist() == [6, 0]
    pages.fork()  # (parents: both 0)
    before = pages.cache.clone()

    def turn():
        pages.want_lens.copy_(pages.kv_lens + 1)
        pages.fit()
        step.block_table.copy_(pages.block_table)
        step.kv_lens.copy_(pages.step_lens)
        step.run()
        pages.advance()

    step.latent.fill_(50.0)
    if captured:
        s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
            turn()
        turn = graph.replay
    for _ in range(3):
        turn()
        torch.cuda.synchronize()
        assert int(pages.status) == abi.DEV_NO_PAGES and int(step.status) == 0
        assert pages.kv_lens.tolist() == [6, 6] and pages.step_lens.tolist() == [0, 0] and pages.refs.tolist() == [2, 2]
        assert torch.equal(pages.cache, before)
        assert (step.out == 0).all() and torch.isneginf(step.lse).all()
    # one branch ends: the other goes on where it was
    if not captured:
        pages.parents.copy_(ints([1, -1]))
        pages.fork()
        pages.status.zero_()
        pages.want_lens.copy_(ints([7, 0]))
        pages.fit()
        step.block_table.copy_(pages.block_table)
        step.kv_lens.copy_(pages.step_lens)
        step.run()
        pages.advance()
        torch.cuda.synchronize()
        assert int(pages.status) == 0 and pages.kv_lens.tolist() == [7, 0] and pages.refs.tolist() == [1, 1]
        before[0, 1, 2, :512], before[0, 1, 2, 512:] = 50.0, 0.0
        assert torch.equal(pages.cache, before)


def test_lengths_that_cannot_be_are_not_taken():
    pages = Pages(1, 9, 4, 3, 2)
    pages.want_lens.copy_(ints([3, 9, 5]))  # the second is longer than its row
    pages.fit()
    pages.advance()
    assert int(pages.status) == abi.DEV_BAD_INDPTR
    assert pages.step_lens.tolist() == [3, 0, 5] and pages.kv_lens.tolist() == [3, 0, 5]
    pages.want_lens.copy_(ints([-1, 2, 0]))
    pages.fit()
    pages.advance()
    assert pages.step_lens.tolist() == [0, 2, 0] and pages.kv_lens.tolist() == [3, 2, 0]


@pytest.mark.parametrize("batch", [1, 5, 300, 600, 1500])
@pytest.mark.parametrize("pages", [64, 6000, 40000])
def test_lengths_of_every_request(batch, pages):
    """In every block size and with several blocks, granted and not."""
    g = torch.Generator()
    g.manual_seed(batch)
    have = torch.randint(0, 40, (batch,), generator=g).int()
    want = have + torch.randint(0, 9, (batch,), generator=g).int()
    want[batch // 2] = -1
    need = int(((want.clamp_min(0) + 3) // 4).sum())
    table = torch.full((batch, 13), -1, dtype=torch.int32, device="cuda")
    refs, held, copies, status = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (pages, batch, 3 * batch, 1))
    ws = torch.empty(abi.mla_pages_fit_workspace_bytes(batch, pages), dtype=torch.uint8, device="cuda")
    lens = torch.full((batch,), 77, dtype=torch.int32, device="cuda")
    zero = torch.zeros_like(held)
    abi.mla_pages_fit(zero, want.cuda(), held, table, refs, 4, copies.view(batch, 3), ws, 0, 0, status, None, lens)
    short = need > pages
    assert int(status) == abi.DEV_BAD_INDPTR | (abi.DEV_NO_PAGES if short else 0)
    assert torch.equal(lens.cpu(), torch.zeros_like(want) if short else want.clamp_min(0))


def test_binding_refuses():
    i = lambda *n: torch.zeros(*n, dtype=torch.int32, device="cuda")  # noqa: E731
    ws = torch.zeros(4096, dtype=torch.uint8, device="cuda")
    two = i(2)
    ok = dict(kv_lens=i(2), want_lens=i(2), held=i(2), block_table=i(2, 5), refs=i(9), page_size=4, copies=i(2, 3), workspace=ws)
    for kw, message in [(dict(step_lens=i(3)), "step_lens must"), (dict(step_lens=i(2).long()), "step_lens must"),
                        (dict(step_lens=i(2).cpu()), "step_lens must be a CUDA"), (dict(step_lens=i(4)[::2]), "step_lens must be contiguous"),
                        (dict(step_lens=two, want_lens=two), "invalid"), (dict(step_lens=two, kv_lens=two), "invalid"),
                        (dict(step_lens=two, held=two), "invalid")]:
        with pytest.raises(abi.MlaTreeError, match=message):
            abi.mla_pages_fit(**{**ok, **kw})
    abi.mla_pages_fit(**ok, step_lens=i(2))
