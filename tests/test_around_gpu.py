"""The calls around the attention as a program makes them: on streams of its
own, side by side, one after another without a wait, and over the same cache."""
import math

import pytest
import torch

import __graft_entry__
from speculative_decode_mla_tree_gb300 import abi
from speculative_decode_mla_tree_gb300.step import AcceptStep, DecodeStep, Pages

import paged_ref as ref

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
SCALE = 1.0 / math.sqrt(192.0)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    __graft_entry__.build()


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def scores(x, k, stream=None):
    t = x.shape[0]
    out = [torch.zeros(t, device="cuda"), torch.zeros(t, device="cuda"), torch.zeros(t, k, dtype=torch.int32, device="cuda"),
           torch.zeros(t, k, device="cuda")]
    torch.cuda.synchronize()
    abi.mla_token_logprobs(x, lse=out[0], entropy=out[1], top_ids=out[2], top_logprobs=out[3], stream=stream)
    return out


def test_side_by_side_on_two_streams():
    """Two calls at once, each on a stream of its own and given by argument, give what each gives alone."""
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    xs = [(torch.randn(n, 90001, generator=g, device="cuda") * 3).to(BF) for n in (3, 700)]
    alone = [scores(x, 9) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[scores(x, 9, s) for x, s in zip(xs, streams)] for _ in range(3)]
    torch.cuda.synchronize()
    for run in got:
        for a, b in zip(run, alone):
            assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_scores_then_walk_then_moves_without_a_wait():
    """Each call takes what the one before it leaves, on one stream, many times over."""
    g = torch.Generator()
    g.manual_seed(2)
    n, b, vocab, page = 12, 40, 30011, 16
    cache = torch.randn(2, 6 * b, page, 576, generator=g).to(BF).cuda()
    step = AcceptStep(cache, [n] * b, 6, vocab, max_accept=n, top_k=3)
    step.block_table.copy_(torch.randperm(6 * b, generator=g).view(b, 6).int())
    parents = torch.tensor([-1] + [max(0, i - 1 - i % 3) for i in range(1, n)]).repeat(b, 1)
    for turn in range(4):
        targets = torch.randint(0, vocab, (b, n), generator=g)
        tokens = torch.where(torch.rand(b, n, generator=g) < 0.8, targets.gather(1, parents.clamp_min(0)),
                             torch.randint(0, vocab, (b, n), generator=g))
        logits = torch.randn(b, n, vocab, generator=g).scatter(2, targets[..., None], 12.0)
        step.logits.copy_(logits.view(b * n, vocab))
        step.parents.copy_(parents.reshape(-1).int())
        step.tokens.copy_(tokens.reshape(-1).int())
        step.first.copy_(tokens[:, 0].int())
        lens = torch.randint(n, 6 * page + 1, (b,), generator=g)
        step.kv_lens.copy_(lens.int())
        want = cache.cpu().clone()
        step.run()
        torch.cuda.synchronize()
        assert int(step.status) == 0
        t = step.block_table.tolist()
        for r in range(b):
            cur, wanted, path = -1, int(tokens[r, 0]), []
            while True:
                good = [i for i in range(n) if parents[r, i] == cur and tokens[r, i] == wanted]
                if not good:
                    break
                cur = good[0]
                path.append(cur)
                wanted = int(targets[r, cur])
            base = int(lens[r]) - n
            for k, i in enumerate(path):
                p, q = base + i, base + k
                want[:, t[r][q // page], q % page] = want[:, t[r][p // page], p % page]
            assert step.path[r].tolist() == path + [-1] * (n - len(path))
            assert int(step.next_tokens[r]) == wanted and int(step.kv_lens[r]) == base + len(path)
        assert torch.equal(cache.cpu(), want)


def test_pages_on_a_stream_of_their_own():
    """Every call of Pages goes to the stream that it is given: what that stream captures does not happen before the replay."""
    pages = Pages(1, 8, 4, 2, 3)
    pages.fit()
    pages.want_lens.copy_(torch.tensor([3, 5]))
    torch.cuda.synchronize()
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        graph.capture_begin(capture_error_mode="relaxed")
    pages.fit(s)
    pages.advance(s)
    with torch.cuda.stream(s):
        graph.capture_end()
    assert pages.kv_lens.tolist() == [0, 0] and pages.held.tolist() == [0, 0]
    graph.replay()
    assert pages.kv_lens.tolist() == [3, 5] and pages.held.tolist() == [1, 2] and int(pages.status) == 0


def test_walk_without_alternatives():
    """Given targets and no alternatives: the step scores the rows alone."""
    cache = torch.zeros(4, 8, 576, dtype=BF, device="cuda")
    targets = torch.tensor([5, 6, 7], dtype=torch.int32, device="cuda")
    step = AcceptStep(cache, [3, 0], 2, 50, top_k=0, targets=targets)
    step.block_table.copy_(torch.tensor([[0, 1], [2, 3]]))
    step.kv_lens.copy_(torch.tensor([7, 0]))
    step.parents.copy_(torch.tensor([-1, 0, 1]))
    step.tokens.copy_(torch.tensor([4, 5, 9]))
    step.first.copy_(torch.tensor([4, 3]))
    step.run()
    assert step.counts.tolist() == [2, 0] and step.next_tokens.tolist() == [6, 3] and step.kv_lens.tolist() == [6, 0]
    assert (step.entropy - math.log(50)).abs().max() < 1e-5 and int(step.status) == 0


def test_walk_by_given_targets():
    """Tokens drawn elsewhere instead of the most likely ones."""
    cache = torch.zeros(4, 8, 576, dtype=BF, device="cuda")
    drawn = ints([7, 8, 9])
    step = AcceptStep(cache, [3], 4, 20, targets=drawn)
    step.parents.copy_(ints([-1, 0, 1]))
    step.tokens.copy_(ints([5, 7, 3]))
    step.first.fill_(5)
    step.kv_lens.fill_(3)
    step.run()
    assert step.counts.tolist() == [2] and step.next_tokens.tolist() == [8] and step.kv_lens.tolist() == [2]


@pytest.mark.parametrize("window,sinks", [(0, 0), (20, 3)])
def test_branches_decode_over_shared_pages(window, sinks):
    """A prompt, four branches of it, tokens appended to each through its own pages, and their
    attention against every branch's own rows; with a window the pages behind it are free again."""
    page, width, heads, batch = 8, 12, 8, 4
    g = torch.Generator()
    g.manual_seed(3)
    pages = Pages(1, 40, page, batch, width, window, sinks)
    cache = pages.cache[0]
    rope = torch.cat([torch.ones(128, 32), torch.zeros(128, 32)], 1).cuda()
    rows = [torch.randn(45, 576, generator=g).to(BF)] + [torch.zeros(0, 576, dtype=BF)] * 3
    pages.want_lens[0] = 45
    pages.fit()
    pages.advance()
    step = DecodeStep(cache, batch, heads, width, rope, SCALE, window=window, sinks=sinks)
    abi.mla_paged_append(rows[0][:, :512].cuda(), rows[0][:, 512:].cuda(), ints([0, 45, 45, 45, 45]), pages.kv_lens, pages.block_table, cache, rope)
    for turn in range(22):
        parents = [0] * batch if turn == 0 else torch.randint(0, batch, (batch,), generator=g).tolist() if turn % 5 == 0 else list(range(batch))
        pages.parents.copy_(ints(parents))
        pages.fork()
        rows = [rows[p] for p in parents]
        pages.want_lens.copy_(pages.kv_lens + 1)
        pages.fit()
        new = torch.randn(batch, 576, generator=g).to(BF)
        rows = [torch.cat([r, n[None]]) for r, n in zip(rows, new)]
        pages.advance()
        step.block_table.copy_(pages.block_table)
        step.kv_lens.copy_(pages.kv_lens)
        step.latent.copy_(new[:, :512])
        step.k_rope.copy_(new[:, 512:])
        q = torch.randn(batch, heads, 576, generator=g).to(BF)
        step.q.copy_(q)
        step.run()
        torch.cuda.synchronize()
        assert int(pages.status) == 0 and int(step.status) == 0
        for b in range(batch):
            n = rows[b].shape[0]
            seen = [j for j in range(n) if not window or j < sinks or j >= n - window]
            wo, wl, to, tl = ref.decode(q[b:b + 1], rows[b][seen], torch.arange(len(seen))[None].int(), [len(seen)], 1, SCALE)
            assert ((step.out[b:b + 1].double().cpu() - wo).abs() <= to).all(), (turn, b)
            assert ((step.lse[b:b + 1].double().cpu() - wl).abs() <= tl).all()
    table, held = pages.block_table.tolist(), pages.held.tolist()
    count = [0] * 40
    for b in range(batch):
        for p in table[b][:held[b]]:
            if p >= 0:
                count[p] += 1
    assert count == pages.refs.tolist()
    if window:  # 67 positions: columns 0 (sinks) and those of the last 20
        assert all(sum(p >= 0 for p in table[b][:held[b]]) <= 1 + 4 for b in range(batch))
