"""A decoding step of a fixed batch shape with slots that hold no request."""

import pytest
import torch

import __graft_entry__
from speculative_decode_mla_tree_gb300 import abi
from speculative_decode_mla_tree_gb300.step import DecodeStep

import paged_ref as ref
from test_paged_gpu import BF, SCALE, check, gen, normal, paged, rope_table

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    __graft_entry__.build()


@pytest.mark.parametrize("page", [16, 3])
def test_step_with_empty_slots(page):
    """Slots come and go in a captured step: an empty one (length 0) sets no
    status bit, writes no cache row, leaves its query alone and gives 0 and -inf."""
    g = gen(80)
    B, heads, width = 6, 8, 40 // page + 1
    rounds = [[0, 20, 0, 1, 33, 0], [7, 21, 0, 0, 34, 0], [0] * 6, [8, 0, 40, 1, 0, 2]]
    cache = torch.full((B * width, page, 576), float("nan"), dtype=BF, device="cuda")
    flat = normal(g, B * width * page, 576)
    cache.copy_(flat.view(cache.shape))
    rope = rope_table(64)
    step = DecodeStep(cache, B, heads, width, rope.cuda(), SCALE)
    table = torch.randperm(B * width, generator=g).int().view(B, width)
    step.run()  # no slot in use
    torch.cuda.synchronize()
    assert int(step.status) == 0
    assert torch.equal(cache.cpu().view(-1, 576), flat)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.run()
    for lens in rounds:
        # an empty slot's entries name no page, or another request's
        shown = torch.where(torch.tensor(lens)[:, None] > 0, table, torch.where(table % 2 == 0, table.flip(0), -1))
        row, q = normal(g, B, 576), normal(g, B, heads, 576)
        step.block_table.copy_(shown)
        step.kv_lens.copy_(torch.tensor(lens))
        step.latent.copy_(row[:, :512])
        step.k_rope.copy_(row[:, 512:])
        step.q.copy_(q)
        graph.replay()
        torch.cuda.synchronize()
        assert int(step.status) == 0
        live = [b for b in range(B) if lens[b]]
        got, turned = cache.cpu().view(-1, 576), step.q.cpu()
        if live:
            pick = torch.tensor(live)
            slots, rows, tol, qs, qtol = ref.append(row[pick, :512], row[pick, 512:], list(range(len(live) + 1)),
                                                    [lens[b] for b in live], table[pick], None, page, rope,
                                                    q[pick][:, :, 512:])
            assert ((got[slots].double() - rows).abs() <= tol).all()
            assert ((turned[pick][:, :, 512:].double() - qs).abs() <= qtol).all()
            flat[slots] = got[slots]
        assert torch.equal(got, flat)
        empty = torch.tensor([b for b in range(B) if not lens[b]])
        assert torch.equal(turned[empty], q[empty])
        assert (step.out[empty.cuda()] == 0).all() and torch.isneginf(step.lse[empty.cuda()]).all()
        check(step.out, step.lse, ref.decode(turned, flat, table, lens, page, SCALE))


def test_step_reports_bad_lengths_beside_empty_slots():
    """What is wrong stays visible: a negative length and one beyond the table."""
    g = gen(81)
    cache = normal(g, 8, 16, 576).cuda()
    before = cache.clone()
    step = DecodeStep(cache, 4, 8, 2, rope_table(64).cuda(), SCALE)
    step.block_table.copy_(torch.arange(8).view(4, 2))
    for bad in (-1, 33, -(1 << 31), (1 << 31) - 1):
        step.status.zero_()
        step.kv_lens.copy_(torch.tensor([0, bad, 0, 5]))
        step.append()
        assert int(step.status) == abi.DEV_BAD_INDPTR
        changed = (cache.view(torch.int16) != before.view(torch.int16)).any(-1).nonzero().tolist()
        assert changed == [[6, 4]]


@pytest.mark.parametrize("batch", [1, 33, 300])
def test_one_token_a_request(batch):
    """qo_indptr None is one token a request: the same rows as with 0, 1, 2, ..."""
    g = gen(82 + batch)
    lens = torch.randint(1, 60, (batch,), generator=g).tolist()
    cache, _, table = paged(g, lens, 16)
    other = cache.clone()
    row, q = normal(g, batch, 576).cuda(), normal(g, batch, 5, 64).cuda()
    pos = torch.randint(0, 64, (batch,), generator=g).int().cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    outs = [torch.zeros_like(q) for _ in range(2)]
    for ptr, c, o in ((None, cache, outs[0]), (torch.arange(batch + 1, dtype=torch.int32, device="cuda"), other, outs[1])):
        abi.mla_paged_append(row[:, :512], row[:, 512:], ptr, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                             table.cuda(), c, rope_table(64).cuda(), q, o, pos, status=status)
    assert torch.equal(cache.view(torch.int16), other.view(torch.int16)) and torch.equal(*outs)
    assert int(status) == 0


def test_one_token_a_request_needs_as_many_tokens():
    """Tokens and requests are one to one, or the call is refused."""
    g = gen(83)
    cache, _, table = paged(g, [5, 6], 16)
    row = normal(g, 3, 576).cuda()
    with pytest.raises(abi.MlaTreeError):
        abi.mla_paged_append(row[:, :512], row[:, 512:], None, torch.tensor([5, 6], dtype=torch.int32, device="cuda"),
                             table.cuda(), cache, rope_table(64).cuda())


@pytest.mark.parametrize("tokens,heads", [(1, 1), (1, 3), (4, 1)])
@pytest.mark.parametrize("in_place", [False, True], ids=["apart", "in_place"])
def test_append_strides_of_single_elements(tokens, heads, in_place):
    """The stride of a dimension of size 1 says nothing: views that differ in
    it alone are the same queries."""
    g = gen(84)
    cache, _, table = paged(g, [tokens], 16)
    row, x = normal(g, tokens, 576).cuda(), normal(g, tokens, heads, 64)
    odd = 64 * heads + (4 if tokens == 1 else 0), 68 if heads == 1 else 64, 1  # no whole 16-byte pieces

    def views(t):
        return t, t.as_strided(t.shape, odd)

    want = torch.zeros_like(x, device="cuda")
    rope, n = rope_table(64).cuda(), torch.tensor([tokens], dtype=torch.int32, device="cuda")
    ptr = torch.tensor([0, tokens], dtype=torch.int32, device="cuda")
    abi.mla_paged_append(row[:, :512], row[:, 512:], ptr, n, table.cuda(), cache, rope, x.cuda(), want)
    for k in range(2):
        for m in range(2):
            q = x.cuda()
            out = q if in_place else torch.zeros_like(q)
            abi.mla_paged_append(row[:, :512], row[:, 512:], ptr, n, table.cuda(), cache, rope, views(q)[k], views(out)[m])
            assert torch.equal(out, want)
