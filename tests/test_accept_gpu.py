"""Tree acceptance and the compaction of accepted rows on the GPU against plain
loops; both move integers and rows, so every comparison is exact."""
import random

import pytest
import torch

import __graft_entry__
from speculative_decode_mla_tree_gb300 import abi
from speculative_decode_mla_tree_gb300.step import AcceptStep

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    __graft_entry__.build()


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def walk(parents, tokens, targets, first, most):
    """(path, next token) of one tree."""
    n, cur, path = len(parents), -1, []
    want = first if first is not None else tokens[0] if n else -1
    while len(path) < most:
        good = [i for i in range(n) if -1 <= parents[i] < i and parents[i] == cur and tokens[i] == want]
        if not good:
            break
        cur = good[0]
        path.append(cur)
        want = targets[cur]
    return path, want


def forest(r, n, vocab, chain=False):
    """Parents in topological order (several roots now and then), tokens and targets of few values, so that walks go on."""
    parents = [i - 1 if chain else -1 if i == 0 or r.random() < 0.1 else r.randrange(max(0, i - 6), i) for i in range(n)]
    return parents, [r.randrange(vocab) for _ in range(n)], [r.randrange(vocab) for _ in range(n)]


def accept(trees, lens, most, first=None, targets=None, status=None, in_place=False):
    indptr, flat = [0], [[], [], []]
    for t in trees:
        indptr.append(indptr[-1] + len(t[0]))
        for a, b in zip(flat, t):
            a.extend(b)
    b = len(trees)
    path = torch.full((b, most), 99, dtype=torch.int32, device="cuda")
    counts, nxt = torch.full((b,), 99, dtype=torch.int32, device="cuda"), torch.full((b,), 99, dtype=torch.int32, device="cuda")
    kv = ints(lens)
    new = kv if in_place else torch.full_like(kv, 99)
    abi.mla_tree_accept(ints(flat[0]), ints(flat[1]), ints(flat[2]) if targets is None else targets, ints(indptr), kv, path,
                        counts, nxt, new, None if first is None else ints(first), status)
    return path.cpu().tolist(), counts.cpu().tolist(), nxt.cpu().tolist(), new.cpu().tolist()


def check_accept(trees, lens, most, first):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = accept(trees, lens, most, first, status=status, in_place=most % 2 == 0)
    for b, t in enumerate(trees):
        path, nxt = walk(*t, None if first is None else first[b], most)
        assert got[0][b] == path + [-1] * (most - len(path)), (b, t)
        assert (got[1][b], got[2][b], got[3][b]) == (len(path), nxt, lens[b] - len(t[0]) + len(path)), (b, t)
    assert int(status) == 0


@pytest.mark.parametrize("seed", range(4))
@pytest.mark.parametrize("most", [0, 1, 3, 16, 200])
def test_accept(seed, most):
    r = random.Random(seed)
    trees = [forest(r, n, 3 if n > 2 else 2) for n in [0, 1, 2, 9, 33, 64, 127, 128, 129, 300, 1, 16, 0]]
    lens = [len(t[0]) + r.randrange(100) for t in trees]
    check_accept(trees, lens, most, None)
    check_accept(trees, lens, most, [r.randrange(3) for _ in trees])


@pytest.mark.parametrize("n", [2047, 2048, 6000, 8192])
def test_long_trees(n):
    """Chains that are taken whole; with more than 6000 nodes the targets stay in device memory."""
    r = random.Random(n)
    p, _, _ = forest(r, n, 1, chain=True)
    trees = [(p, [7] * n, [7] * n), forest(r, n, 2), (p, [7] * n, [7] * (n // 2) + [8] * (n - n // 2))]
    check_accept(trees, [n, n + 5, n + 1], n, [7, 0, 7])
    check_accept(trees, [n, n + 5, n + 1], 20, None)


def test_equal_siblings_and_many_requests():
    r = random.Random(5)
    same = ([-1, -1, 0, 0, 1, 1], [4, 4, 5, 5, 5, 5], [5, 5, 9, 9, 9, 9])
    check_accept([same], [6], 4, [4])     # the lowest of equal children, and never the other's
    trees = [forest(r, r.randrange(0, 40), 2) for _ in range(1500)]
    check_accept(trees, [len(t[0]) + 3 for t in trees], 12, [0] * 1500)


def test_next_tokens_over_first():
    """A loop that keeps one buffer for the tokens to go on with."""
    r = random.Random(8)
    trees = [forest(r, n, 2) for n in (9, 0, 300, 1)]
    n = [len(t[0]) for t in trees]
    flat = [ints([x for t in trees for x in t[i]]) for i in range(3)]
    keep = ints([1, 1, 0, 1])
    path, counts = torch.zeros(4, 6, dtype=torch.int32, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    abi.mla_tree_accept(*flat, ints([0, n[0], n[0], n[0] + n[2], sum(n)]), ints(n), path, counts, keep, counts.clone(), first=keep)
    want = [walk(*t, f, 6) for t, f in zip(trees, (1, 1, 0, 1))]
    assert keep.tolist() == [w[1] for w in want] and counts.tolist() == [len(w[0]) for w in want]


def test_targets_of_any_stride():
    r = random.Random(6)
    t = forest(r, 50, 2)
    wide = torch.zeros(50, 5, dtype=torch.int32, device="cuda")
    wide[:, 3] = ints(t[2])
    got = accept([t], [60], 8, targets=wide[:, 3])
    path, nxt = walk(*t, None, 8)
    assert got[0][0][:len(path)] == path and got[2] == [nxt]


def test_accept_bad_input():
    good = ([-1, 0, 1], [1, 1, 1], [1, 1, 1])
    st = lambda: torch.zeros(1, dtype=torch.int32, device="cuda")  # noqa: E731
    s = st()
    got = accept([good, ([-1, 1, 5], [1, 1, 1], [1, 1, 1]), good], [3, 3, 3], 4, status=s)
    assert int(s) == abi.DEV_BAD_PARENT and got[1] == [3, 1, 3]
    s = st()
    got = accept([good, good], [3, 2], 4, status=s)           # more nodes than positions
    assert int(s) == abi.DEV_BAD_INDPTR and got[1] == [3, 0] and got[2] == [1, -1] and got[3] == [3, 2]
    assert got[0][1] == [-1] * 4
    s = st()
    n = 8193
    big = (list(range(-1, n - 1)), [1] * n, [1] * n)
    got = accept([big, good], [n, 3], 4, status=s)
    assert int(s) == abi.DEV_TREE_TOO_BIG and got[1] == [0, 3] and got[3] == [n, 3]
    for bad in ([0, 3, 2], [0, 2, 4], [-1, 2, 3]):
        s = st()
        path, c = torch.zeros(2, 2, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
        abi.mla_tree_accept(ints(good[0]), ints(good[1]), ints(good[2]), ints(bad), ints([9, 9]), path, c, c.clone(), c.clone(),
                            status=s)
        assert int(s) & abi.DEV_BAD_INDPTR


# --------------------------------------------------------------- compaction

def caches(r, layers, pages, page, gap, layer_gap):
    """A cache [layers, pages, page, 576] with holes between its pages and layers, and a CPU copy of it."""
    g = torch.Generator()
    g.manual_seed(r.randrange(1 << 30))
    each = pages * (page * 576 + gap) + layer_gap
    store = torch.randn(layers, each, generator=g).to(BF).cuda()
    cache = store[:, :pages * (page * 576 + gap)].unflatten(1, (pages, page * 576 + gap))[:, :, :page * 576].unflatten(2, (page, 576))
    return store, cache


def moved(cache, table, page, lens, counts, paths):
    want = cache.cpu().clone()
    for b, path in enumerate(paths):
        base = lens[b] - counts[b]
        for k in range(counts[b]):
            p, q = base + path[k], base + k
            want[:, table[b][q // page], q % page] = want[:, table[b][p // page], p % page]
    return want


@pytest.mark.parametrize("layers,page,gap,layer_gap", [(1, 64, 0, 0), (2, 16, 0, 8), (5, 8, 24, 0), (9, 3, 8, 64), (4, 1, 0, 0)])
def test_compact(layers, page, gap, layer_gap):
    r = random.Random(layers * page)
    sizes = [1, 1, 5, 9, 64, 130, 200, 17]
    base = [r.randrange(0, 100) for _ in sizes]
    used = [-(-(b + n) // page) for b, n in zip(base, sizes)]
    order = list(range(sum(used) + 2))
    r.shuffle(order)
    table, at = [], 0
    for u in used:
        table.append(order[at:at + u])
        at += u
    paths = [sorted(r.sample(range(n), r.randrange(0, n + 1))) for n in sizes]
    paths[4] = list(range(64))                   # nothing moves
    paths[5] = [0] + list(range(2, 130))         # every row but the first moves up by one
    paths[6] = list(range(60, 200))              # more than two rounds, all by the same distance
    counts = [len(p) for p in paths]
    lens = [b + c for b, c in zip(base, counts)]
    store, cache = caches(r, layers, at + 2, page, gap, layer_gap)
    before = store.cpu().clone()
    want = moved(cache, table, page, lens, counts, paths)
    width = max(used)
    path = ints([p + [-1] * (201 - len(p)) for p in paths])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    c = cache if layers > 1 else cache[0]
    abi.mla_paged_compact(path, ints(counts), ints(lens), ints([t + [-9] * (width - len(t)) for t in table]), c, status)
    assert torch.equal(cache.cpu(), want) and int(status) == 0
    after = store.cpu()
    hole = torch.ones_like(before, dtype=torch.bool)
    hole[:, :(at + 2) * (page * 576 + gap)].unflatten(1, (at + 2, page * 576 + gap))[:, :, :page * 576] = False
    assert torch.equal(after[hole].view(torch.int16), before[hole].view(torch.int16))


def test_compact_layers_inside_pages():
    """[pages, layers, page, 576] in memory, seen as [layers, pages, page, 576]."""
    g = torch.Generator()
    g.manual_seed(4)
    store = torch.randn(6, 5, 8, 576, generator=g).to(BF).cuda()
    cache = store.transpose(0, 1)
    table, path = [[3, 1, 0]], [[0, 2, 7, 12]]
    want = moved(cache, table, 8, [9], [4], path)
    abi.mla_paged_compact(ints(path), ints([4]), ints([9]), ints(table), cache)
    assert torch.equal(cache.cpu(), want)
    with pytest.raises(abi.MlaTreeError, match="invalid"):
        abi.mla_paged_compact(ints(path), ints([4]), ints([9]), ints(table), store[:, :1].transpose(0, 1).expand(3, 6, 8, 576))


def test_compact_bad_input():
    page, table = 4, [[0, 1, 2], [3, 77, 5], [6, 7, 8]]
    g = torch.Generator()
    g.manual_seed(1)
    cache = torch.randn(9, page, 576, generator=g).to(BF).cuda()
    before = cache.cpu().clone()
    for path, counts, lens, bit, ok in [
            ([[1, 3, 2, 5]] * 3, [4, 0, 0], [6, 0, 0], abi.DEV_BAD_PARENT, 2),       # stops before the node that goes back
            ([[2, 2, 3, 5]] * 3, [4, 0, 0], [6, 0, 0], abi.DEV_BAD_PARENT, 1),
            ([[1, 3, 11, 12]] * 3, [4, 0, 0], [6, 0, 0], abi.DEV_BAD_PARENT, 2),     # a position behind the table
            ([[-1, 3, 5, 6]] * 3, [4, 0, 0], [6, 0, 0], abi.DEV_BAD_PARENT, 0),
            ([[1, 3, 4, 5]] * 3, [5, 0, 0], [6, 0, 0], abi.DEV_BAD_INDPTR, 0),
            ([[1, 3, 4, 5]] * 3, [4, 0, 0], [3, 0, 0], abi.DEV_BAD_INDPTR, 0),
            ([[1, 3, 4, 5]] * 3, [4, 0, 0], [13, 0, 0], abi.DEV_BAD_INDPTR, 0),
            ([[1, 3, 4, 5]] * 3, [-1, 0, 0], [6, 0, 0], abi.DEV_BAD_INDPTR, 0)]:
        cache.copy_(before)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        abi.mla_paged_compact(ints(path), ints(counts), ints(lens), ints(table), cache, status)
        want = moved(before[None], table, page, [lens[0] - counts[0] + ok, 0, 0], [ok, 0, 0], path)[0] if ok else before
        assert torch.equal(cache.cpu(), want) and int(status) == bit, (path, counts, lens)
    # rows 1 and 6 of request 1 lie in its bad page: only the moves that touch it are left out
    cache.copy_(before)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    abi.mla_paged_compact(ints([[0, 0, 0]] * 1 + [[1, 4, 8]] + [[0, 0, 0]]), ints([0, 3, 0]), ints([0, 3, 0]), ints(table), cache, status)
    want = before.clone()
    want[3, 0], want[3, 2] = before[3, 1], before[5, 0]
    assert torch.equal(cache.cpu(), want) and int(status) == abi.DEV_BAD_SLOT


def test_step_in_a_graph():
    """Logits to moved rows, captured once and replayed on other contents."""
    r = random.Random(9)
    vocab, page, layers, b, n = 50, 8, 3, 4, 7
    g = torch.Generator()
    g.manual_seed(9)
    cache = torch.randn(layers, 24, page, 576, generator=g).to(BF).cuda()
    step = AcceptStep(cache, [n] * b, 6, vocab, max_accept=5)
    perm = torch.randperm(24, generator=g).int().view(b, 6)
    step.block_table.copy_(perm)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            step.run()
    torch.cuda.synchronize()
    for i in range(4):
        trees = [forest(r, n, 3) for _ in range(b)]
        logits = torch.randn(b * n, vocab, generator=g).to(BF)
        for t, tree in enumerate(trees):
            for j in range(n):
                logits[t * n + j, tree[2][j]] = 20.0
        lens = [n + r.randrange(0, 30) for _ in range(b)]
        first = [tree[1][0] for tree in trees]
        step.parents.copy_(torch.tensor([p for t in trees for p in t[0]], dtype=torch.int32))
        step.tokens.copy_(torch.tensor([p for t in trees for p in t[1]], dtype=torch.int32))
        step.first.copy_(torch.tensor(first, dtype=torch.int32))
        step.kv_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        step.logits.copy_(logits)
        want = [walk(*t, f, 5) for t, f in zip(trees, first)]
        counts = [len(w[0]) for w in want]
        new = [ln - n + c for ln, c in zip(lens, counts)]
        rows = moved(cache, perm.tolist(), page, new, counts, [w[0] for w in want])
        graph.replay()
        torch.cuda.synchronize()
        assert step.counts.tolist() == counts and step.next_tokens.tolist() == [w[1] for w in want]
        assert step.kv_lens.tolist() == new and torch.equal(cache.cpu(), rows)
        lp = torch.log_softmax(logits.double(), -1)
        best = lp.max(-1)
        assert (step.top_logprobs[:, 0].cpu().double() - best.values).abs().max() < 1e-4
        assert torch.equal(step.top_ids[:, 0].cpu().long(), best.indices)
        assert (step.entropy.cpu().double() + (lp.exp() * lp).sum(-1)).abs().max() < 1e-4
    assert int(step.status) == 0


def test_binding_refuses():
    i = lambda *n: torch.zeros(*n, dtype=torch.int32, device="cuda")  # noqa: E731
    ok = dict(parents=i(6), tokens=i(6), targets=i(6), qo_indptr=i(3), kv_lens=i(2), path=i(2, 4), counts=i(2),
              next_tokens=i(2), new_lens=i(2))
    for kw, message in [(dict(parents=i(6).cpu()), "parents must be a CUDA"), (dict(tokens=i(5)), "tokens must"),
                        (dict(tokens=i(12)[::2]), "tokens must be contiguous"), (dict(targets=i(6).long()), "targets must"),
                        (dict(qo_indptr=i(2)), "qo_indptr must"), (dict(kv_lens=i(3)), "kv_lens must"),
                        (dict(path=i(8)), "path must"), (dict(counts=i(1)), "counts must"), (dict(first=i(3)), "first must"),
                        (dict(next_tokens=i(2).float()), "next_tokens must"), (dict(status=i(2).float()), "status must")]:
        with pytest.raises(abi.MlaTreeError, match=message):
            abi.mla_tree_accept(**{**ok, **kw})
    cache = torch.zeros(2, 3, 4, 576, dtype=BF, device="cuda")
    ok = dict(path=i(2, 4), counts=i(2), kv_lens=i(2), block_table=i(2, 3), cache=cache)
    for kw, message in [(dict(cache=cache[..., :512]), "cache must"), (dict(cache=cache.transpose(1, 2)), "cache must"),
                        (dict(cache=cache.float()), "cache must"), (dict(path=i(3, 4)), "path must"),
                        (dict(counts=i(3)), "counts must"), (dict(block_table=i(6)), "block_table must"),
                        (dict(kv_lens=i(2).cpu()), "kv_lens must be a CUDA")]:
        with pytest.raises(abi.MlaTreeError, match=message):
            abi.mla_paged_compact(**{**ok, **kw})
