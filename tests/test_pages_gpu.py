"""Forking, fitting and copying pages on the GPU against plain loops over the
same rules; all of it integers and moved rows, compared exactly."""
import random

import pytest
import torch

import __graft_entry__
from speculative_decode_mla_tree_gb300 import abi
from speculative_decode_mla_tree_gb300.step import Pages

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    __graft_entry__.build()


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Model:
    """The rules, a page at a time."""

    def __init__(self, pages, page, batch, width):
        self.refs, self.page, self.width = [0] * pages, page, width
        self.rows = [[-1] * width for _ in range(batch)]   # behind held: -1, which the calls need not write
        self.held, self.lens = [0] * batch, [0] * batch

    def fork(self, parents):
        children = [parents.count(s) for s in range(len(self.rows))]
        for s, row in enumerate(self.rows):
            for p in row[:self.held[s]]:
                if p >= 0:
                    self.refs[p] += children[s] - 1
        self.rows = [list(self.rows[p][:self.held[p]]) + [-1] * (self.width - self.held[p]) if p >= 0 else [-1] * self.width
                     for p in parents]
        self.held = [self.held[p] if p >= 0 else 0 for p in parents]
        self.lens = [self.lens[p] if p >= 0 else 0 for p in parents]

    def fit(self, want, window=0, sinks=0):
        """The copies, or None where the pages do not suffice."""
        ps, refs = self.page, list(self.refs)
        rows, back, mark = [list(r) for r in self.rows], [], []
        for b, row in enumerate(rows):
            need, n = -(-want[b] // ps), self.lens[b]
            back += [(b, c) for c in range(need, self.held[b]) if row[c] >= 0]
            if window and n + 1 > window:
                for c in range(min((n + 1 - window) // ps, self.held[b], need) - 1, -(-sinks // ps) - 1, -1):
                    if row[c] == -1:
                        break
                    back.append((b, c))
            mark += [(b, c) for c in range(n // ps, min(need, self.held[b])) if want[b] > n and row[c] >= 0 and self.refs[row[c]] > 1]
        for b, c in back + mark:
            refs[rows[b][c]] -= 1
        keep = {}
        for b, c in mark:
            if refs[rows[b][c]] == 0:
                keep.setdefault(rows[b][c], (b, c))
        for p in keep:
            refs[p] = 1
        for b, c in back:
            rows[b][c] = -1
        free = iter([p for p, r in enumerate(refs) if r == 0])
        copies = []
        try:
            for b, row in enumerate(rows):
                need, n = -(-want[b] // ps), self.lens[b]
                copy = (-1, -1, 0)
                for c in range(self.held[b], min(n // ps, need) if want[b] > n else need):
                    row[c] = -1
                for c in range(n // ps, need if want[b] > n else 0):
                    shared = (b, c) in mark and keep.get(row[c]) != (b, c)
                    if c >= self.held[b] or row[c] < 0 or shared:
                        old, row[c] = row[c], next(free)
                        refs[row[c]] = 1
                        if shared and c == n // ps and n % ps:
                            copy = (old, row[c], n % ps)
                copies.append(copy)
        except StopIteration:
            return None
        self.refs, self.rows = refs, rows
        self.held = [-(-w // ps) for w in want]
        return copies


def state(m):
    return ints(m.rows), ints(m.held), ints(m.lens), ints(m.refs)


def same(m, table, held, refs):
    assert held.tolist() == m.held
    assert refs.tolist() == m.refs
    t = table.cpu().tolist()
    for b, h in enumerate(m.held):
        assert t[b][:h] == m.rows[b][:h], b
    count = [0] * len(m.refs)
    for b, h in enumerate(m.held):
        for p in t[b][:h]:
            if p >= 0:
                count[p] += 1
    assert count == m.refs  # nothing is lost and nothing held twice


def fit(m, table, held, lens, refs, want, window=0, sinks=0):
    copies = torch.full((len(want), 3), 55, dtype=torch.int32, device="cuda")
    ws = torch.full((abi.mla_pages_fit_workspace_bytes(len(want), len(m.refs)),), 255, dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    abi.mla_pages_fit(lens, ints(want), held, table, refs, m.page, copies, ws, window, sinks, status)
    return copies.cpu().tolist(), int(status)


@pytest.mark.parametrize("batch,page,width,pages", [(1, 1, 40, 50), (3, 4, 30, 90), (8, 16, 12, 70), (40, 8, 20, 500),
                                                    (65, 64, 9, 400), (300, 4, 9, 2000), (20, 8, 16, 40000),
                                                    (1300, 4, 9, 9000), (2100, 2, 40, 50000)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (9, 2), (30, 17)])
def test_lives_of_branches(batch, page, width, pages, window, sinks):
    """Prompts, single tokens, forks, drops, cuts and reorderings by chance, every state compared."""
    r = random.Random(batch * 100 + window)
    m = Model(pages, page, batch, width)
    table, held, lens, refs = state(m)
    most = width * page
    short = 0
    for turn in range(14):
        kind = r.choice(["grow", "grow", "one", "one", "fork", "cut", "none"])
        if kind == "fork":
            near = r.random() < 0.5
            parents = [r.choice([-1, b, b, b // 4 * 4 if near else r.randrange(batch)]) for b in range(batch)]
            new = torch.full_like(table, -1), torch.full_like(held, 9), torch.full_like(lens, 9)
            status = torch.zeros(1, dtype=torch.int32, device="cuda")
            abi.mla_pages_fork(ints(parents), lens, held, table, refs, new[2], new[1], new[0], status)
            m.fork(parents)
            table, held, lens = new
            assert lens.tolist() == m.lens and int(status) == 0
        else:
            if kind == "cut":  # back to an earlier length, which may lie in a shared page
                m.lens = [r.randrange(0, n + 1) for n in m.lens]
                lens = ints(m.lens)
            top = {"grow": 3 * page, "one": 1, "cut": 2, "none": 0}[kind]
            want = [min(most, n + r.randrange(0, top + 1)) for n in m.lens]
            before = table.cpu().clone(), held.cpu().clone(), refs.cpu().clone()
            copies, status = fit(m, table, held, lens, refs, want, window, sinks)
            expect = m.fit(want, window, sinks)
            if expect is None:
                short += 1
                assert status == abi.DEV_NO_PAGES and copies == [[-1, -1, 0]] * batch
                assert torch.equal(table.cpu(), before[0]) and torch.equal(held.cpu(), before[1]) and torch.equal(refs.cpu(), before[2])
            else:
                assert status == 0 and copies == [list(c) for c in expect]
                m.lens = want
                lens = ints(want)
        same(m, table, held, refs)


def test_all_writers_share_a_page():
    """Of three that hold a page and write to it the lowest keeps it; of two of three, none does."""
    m = Model(10, 8, 3, 4)
    m.rows = [[0, 1, -1, -1]] * 3
    m.refs = [3, 3] + [0] * 8
    m.held, m.lens = [2] * 3, [12] * 3
    table, held, lens, refs = state(m)
    copies, status = fit(m, table, held, lens, refs, [13, 13, 13])
    assert status == 0 and copies == [[-1, -1, 0], [1, 2, 4], [1, 3, 4]]
    assert table.tolist()[0][:2] == [0, 1] and table.tolist()[1][:2] == [0, 2] and table.tolist()[2][:2] == [0, 3]
    assert refs.tolist()[:4] == [3, 1, 1, 1]
    table, held, lens, refs = state(m)
    copies, status = fit(m, table, held, lens, refs, [13, 12, 13])
    assert copies == [[1, 2, 4], [-1, -1, 0], [1, 3, 4]] and refs.tolist()[:4] == [3, 1, 1, 1]


@pytest.mark.parametrize("columns", [2, 20])
def test_a_page_twice_in_a_row_is_kept_once(columns):
    """Entries count, not requests: whoever keeps a page keeps it in one column."""
    m = Model(64, 4, 2, columns)
    m.rows = [[7 if c in (0, columns - 1) else 20 + c for c in range(columns)] for _ in range(2)]
    for row in m.rows:
        for p in row:
            m.refs[p] += 1
    m.held, m.lens = [columns] * 2, [0] * 2
    table, held, lens, refs = state(m)
    copies, status = fit(m, table, held, lens, refs, [4 * columns] * 2)
    assert status == 0 and held.tolist() == [columns] * 2
    rows = table.tolist()
    assert sorted(rows[0])[0] == 0 and sum(row.count(7) for row in rows) == 1 and 7 in rows[0]
    assert len(set(rows[0] + rows[1])) == 2 * columns
    assert refs.tolist() == [int(p in rows[0] + rows[1]) for p in range(64)]


@pytest.mark.parametrize("batch", [3, 300, 600])
@pytest.mark.parametrize("more", [0, 1, 2, 3, 29, 8192 * 2 + 5])
@pytest.mark.parametrize("off", [0, 1])
def test_pools_of_any_size_and_address(batch, more, off):
    """Branches that all write to a shared page and need another one, in pools that are just as large."""
    m = Model(2 + 2 * batch + more, 4, batch, 5)
    store = torch.zeros(len(m.refs) + off, dtype=torch.int32, device="cuda")
    m.rows = [[0, 1, -1, -1, -1] for _ in range(batch)]
    m.refs[0], m.refs[1] = batch, batch
    m.held, m.lens = [2] * batch, [6] * batch
    table, held, lens, refs = state(m)
    refs = store[off:].copy_(refs)
    for want in [[6] * batch, [7] * batch, [9] * batch, [10] * batch]:
        copies, status = fit(m, table, held, lens, refs, want)
        assert status == 0 and copies == [list(c) for c in m.fit(want)]
        m.lens = want
        lens = ints(want)
        same(m, table, held, refs)


def test_exactly_enough_and_one_too_few():
    m = Model(6, 4, 2, 5)
    table, held, lens, refs = state(m)
    copies, status = fit(m, table, held, lens, refs, [12, 13])
    assert status == abi.DEV_NO_PAGES and held.tolist() == [0, 0] and refs.tolist() == [0] * 6
    copies, status = fit(m, table, held, lens, refs, [12, 12])
    assert status == 0 and table.tolist()[0][:3] == [0, 1, 2] and table.tolist()[1][:3] == [3, 4, 5]
    # what one gives back the other takes in the same call
    m.fit([12, 12])
    m.lens = [4, 12]
    lens = ints(m.lens)
    copies, status = fit(m, table, held, lens, refs, [4, 20])
    assert status == 0 and held.tolist() == [1, 5] and table.tolist()[1][:5] == [3, 4, 5, 1, 2]


@pytest.mark.parametrize("batch,columns", [(2, 1 << 30), (7, 300_000_000)])
def test_needs_that_add_up_past_32_bits(batch, columns):
    """Rows that all ask for more pages than there can be: a shortage like any other, and nothing is written."""
    table = torch.empty(batch, columns, dtype=torch.int32, device="cuda")
    refs, held, status = torch.zeros(64, dtype=torch.int32, device="cuda"), ints([0] * batch), ints([0])
    copies = torch.full((batch, 3), 5, dtype=torch.int32, device="cuda")
    ws = torch.empty(abi.mla_pages_fit_workspace_bytes(batch, 64), dtype=torch.uint8, device="cuda")
    abi.mla_pages_fit(ints([0] * batch), ints([columns] * batch), held, table, refs, 1, copies, ws, 0, 0, status)
    assert int(status) == abi.DEV_NO_PAGES
    assert held.tolist() == [0] * batch and refs.tolist() == [0] * 64 and copies.tolist() == [[-1, -1, 0]] * batch


def test_many_pages():
    """More pages than a block counts at a time, free ones far from the front."""
    m = Model(300000, 16, 5, 200)
    m.refs = [1] * 299000 + [0] * 1000
    table, held, lens, refs = state(m)
    copies, status = fit(m, table, held, lens, refs, [3200, 16, 0, 3000, 1])
    assert status == 0
    n = [200, 1, 0, 188, 1]
    at = 299000
    for b in range(5):
        assert table.tolist()[b][:n[b]] == list(range(at, at + n[b]))
        at += n[b]
    assert int(refs.sum()) == 299000 + sum(n)


def test_fork_of_other_sizes():
    """More and fewer rows than before, none at all, tables of other strides."""
    r = random.Random(3)
    m = Model(60, 4, 4, 6)
    assert m.fit([9, 0, 24, 5]) is not None
    m.lens = [9, 0, 24, 5]
    for parents in ([2, 2, 0, -1, 3, 3, 3, 1, 0], [2], [0, 0], [-1, -1, -1], []):
        old = len(m.rows)
        wide = torch.full((old, 11), 123, dtype=torch.int32, device="cuda")
        wide[:, :6] = ints(m.rows).view(old, 6)
        held, lens, refs = ints(m.held), ints(m.lens), ints(m.refs)
        new = torch.full((len(parents), 9), 456, dtype=torch.int32, device="cuda")
        z = lambda: torch.zeros(len(parents), dtype=torch.int32, device="cuda")  # noqa: E731
        nh, nl = z(), z()
        abi.mla_pages_fork(ints(parents), lens, held, wide[:, :6], refs, nl, nh, new[:, :6])
        m.fork(parents)
        same(m, new[:, :6], nh, refs)
        assert nl.tolist() == m.lens and (new[:, 6:] == 456).all()
    assert sum(m.refs) == 0
    big = [r.randrange(0, 40) for _ in range(700)]  # more children than a block looks at at a time
    m = Model(200, 4, 40, 5)
    m.fit([r.randrange(0, 21) for _ in range(40)])
    t, h, ln, refs = state(m)
    nt, nh, nl = torch.full((700, 5), -1, dtype=torch.int32, device="cuda"), torch.zeros(700, dtype=torch.int32, device="cuda"), torch.zeros(
        700, dtype=torch.int32, device="cuda")
    abi.mla_pages_fork(ints(big), ln, h, t, refs, nl, nh, nt)
    m.fork(big)
    same(m, nt, nh, refs)


def test_bad_input():
    m = Model(10, 4, 3, 4)
    m.fit([9, 5, 3])
    table, held, lens, refs = state(m)
    st = lambda: torch.zeros(1, dtype=torch.int32, device="cuda")  # noqa: E731
    new = torch.full((3, 4), -5, dtype=torch.int32, device="cuda"), torch.zeros_like(held), torch.zeros_like(lens)
    s = st()
    abi.mla_pages_fork(ints([0, 3, -2]), lens, held, table, refs, new[2], new[1], new[0], s)
    assert int(s) == abi.DEV_BAD_PARENT and new[1].tolist() == [3, 0, 0] and refs.tolist() == [1, 1, 1] + [0] * 7
    table, held, lens, refs = state(m)
    s, h = st(), ints([3, 5, 1])
    abi.mla_pages_fork(ints([0, 1, 2]), lens, h, table, refs, new[2], new[1], new[0], s)
    assert int(s) == abi.DEV_BAD_INDPTR and new[1].tolist() == [3, 0, 1] and refs.tolist() == m.refs
    s = st()
    t = table.clone()
    t[0, 1] = 10
    abi.mla_pages_fork(ints([1, 1, 2]), lens, held, t, refs, new[2], new[1], new[0], s)
    assert int(s) == abi.DEV_BAD_SLOT and refs.tolist() == [0, 1, 0, 2, 2, 1, 0, 0, 0, 0]
    # lengths that cannot be: those requests stay as they are
    table, held, lens, refs = state(m)
    copies = torch.zeros(3, 3, dtype=torch.int32, device="cuda")
    ws = torch.zeros(abi.mla_pages_fit_workspace_bytes(3, 10), dtype=torch.uint8, device="cuda")
    s = st()
    abi.mla_pages_fit(ints([9, 5, -1]), ints([17, 9, 3]), held, table, refs, 4, copies, ws, status=s)
    assert int(s) == abi.DEV_BAD_INDPTR and held.tolist() == [3, 3, 1] and copies.tolist() == [[-1, -1, 0]] * 3
    assert table[1].tolist()[:3] == [3, 4, 6]
    # page numbers that are none count as missing
    table, held, lens, refs = state(m)
    table[1, 1] = 77
    s = st()
    abi.mla_pages_fit(ints([9, 5, 3]), ints([9, 6, 3]), held, table, refs, 4, copies, ws, status=s)
    assert int(s) == abi.DEV_BAD_SLOT and table[1].tolist()[:2] == [3, 6]


@pytest.mark.parametrize("layers,page,gap", [(1, 64, 0), (3, 16, 8), (7, 1, 0), (2, 200, 0)])
def test_copy(layers, page, gap):
    g = torch.Generator()
    g.manual_seed(page)
    pages = 23
    store = torch.randn(layers, pages, page * 576 + gap, generator=g).to(BF).cuda()
    cache = store[:, :, :page * 576].unflatten(2, (page, 576))
    want = store.cpu().clone()
    entries = [(0, 9, page), (1, 10, 1), (0, 11, page // 2), (2, -1, page), (-1, -1, 0), (3, 12, 0), (4, 13, page - 1),
               (30, 14, 1), (5, 30, 1), (-2, 15, 1), (6, 16, page + 1), (7, 17, -1), (22, 18, page)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    abi.mla_paged_copy(ints(entries), cache if layers > 1 else cache[0], status)
    for s, d, n in entries:
        if 0 <= s < pages and 0 <= d < pages and 0 <= n <= page:
            want[:, d, :n * 576] = want[:, s, :n * 576]
    assert torch.equal(store.cpu().view(torch.int16), want.view(torch.int16)) and int(status) == abi.DEV_BAD_SLOT
    abi.mla_paged_copy(ints(entries)[:0], cache)


def test_beam_search_over_pages_in_a_graph():
    """step.Pages: beams reorder, write a token each and are read again; the rows of every beam are followed by hand."""
    r = random.Random(2)
    page, layers, beams, width = 4, 2, 4, 12
    pool = Pages(layers, 40, page, beams, width)
    rows = [[] for _ in range(beams)]  # the number that stands in each position's row

    def write(first):
        for b in range(beams):
            for j in range(first[b], len(rows[b])):
                t = pool.block_table[b].tolist()
                pool.cache[:, t[j // page], j % page] = rows[b][j]

    def check():
        torch.cuda.synchronize()
        t, c = pool.block_table.cpu().tolist(), pool.cache[:, :, :, 0].cpu()
        for b in range(beams):
            got = [float(c[0, t[b][j // page], j % page]) for j in range(len(rows[b]))]
            assert got == rows[b] and torch.equal(c[0], c[1])
        assert int(pool.status) == 0

    pool.want_lens.copy_(torch.tensor([6, 6, 6, 6], dtype=torch.int32))
    pool.fit()
    rows = [[float(b * 10 + j) for j in range(6)] for b in range(beams)]
    write([0] * beams)
    pool.advance()
    check()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            pool.fork()
            pool.want_lens.copy_(pool.kv_lens + 1)
            pool.fit()
            pool.fork()  # a second one brings the tables back to where the capture found them
            pool.want_lens.copy_(pool.kv_lens + 1)
            pool.fit()
    torch.cuda.synchronize()
    for turn in range(9):
        parents = [r.choice([0, 1, 2, 3]) for _ in range(beams)] if turn else [0, 0, 0, 0]
        pool.parents.copy_(torch.tensor(parents, dtype=torch.int32))
        graph.replay()  # forks twice by the same parents; the first fork's new token is not kept
        for _ in range(2):
            rows = [list(rows[p]) for p in parents]
        for b in range(beams):
            rows[b].append(float(100 + turn * 10 + b))
        write([len(x) - 1 for x in rows])
        pool.advance()
        check()


def test_binding_refuses():
    i = lambda *n: torch.zeros(*n, dtype=torch.int32, device="cuda")  # noqa: E731
    ok = dict(parents=i(3), kv_lens=i(2), held=i(2), block_table=i(2, 5), refs=i(9), new_lens=i(3), new_held=i(3), new_table=i(3, 5))
    for kw, message in [(dict(refs=i(9).cpu()), "refs must be a CUDA"), (dict(refs=i(18)[::2]), "refs must be contiguous"),
                        (dict(parents=i(2)), "parents must"), (dict(kv_lens=i(3)), "kv_lens must"), (dict(held=i(2).long()), "held must"),
                        (dict(new_table=i(3, 4)), "new_table must"), (dict(new_held=i(2)), "new_held must"),
                        (dict(block_table=i(5)), "block_table must"), (dict(status=i(1).float()), "status must")]:
        with pytest.raises(abi.MlaTreeError, match=message):
            abi.mla_pages_fork(**{**ok, **kw})
    t, two = i(4, 5), i(2)
    for kw in (dict(block_table=t[:2], new_table=t[1:]), dict(kv_lens=two, new_lens=two, parents=i(2), new_held=i(2), new_table=i(2, 5)),
               dict(held=two, new_held=two, parents=i(2), new_lens=i(2), new_table=i(2, 5))):
        with pytest.raises(abi.MlaTreeError, match="invalid"):
            abi.mla_pages_fork(**{**ok, **kw})
    ws = torch.zeros(4096, dtype=torch.uint8, device="cuda")
    ok = dict(kv_lens=i(2), want_lens=i(2), held=i(2), block_table=i(2, 5), refs=i(9), page_size=4, copies=i(2, 3), workspace=ws)
    for kw, message in [(dict(want_lens=i(3)), "want_lens must"), (dict(copies=i(2, 2)), "copies must"), (dict(page_size=0), "invalid"),
                        (dict(page_size=1.5), "page_size must"), (dict(window=-1), "invalid"), (dict(sinks=1 << 31), "sinks must"),
                        (dict(workspace=ws[:8]), "workspace"), (dict(workspace=ws[4:]), "workspace"), (dict(refs=i(9).cpu()), "refs must")]:
        with pytest.raises(abi.MlaTreeError, match=message):
            abi.mla_pages_fit(**{**ok, **kw})
    cache = torch.zeros(3, 4, 576, dtype=BF, device="cuda")
    for kw, message in [(dict(copies=i(2, 2)), "copies must"), (dict(copies=i(2, 3).cpu()), "copies must be a CUDA"),
                        (dict(cache=cache[0]), "cache must"), (dict(cache=cache.half()), "cache must")]:
        with pytest.raises(abi.MlaTreeError, match=message):
            abi.mla_paged_copy(**{**dict(copies=i(2, 3), cache=cache), **kw})
