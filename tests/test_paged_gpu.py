"""The paged operators on the GPU against their formulas in 64 bits
(paged_ref), at the sizes, page sizes, head counts and lengths where they can
go wrong; rows that no request owns hold NaN, so that reading one shows."""
import math

import pytest
import torch

import __graft_entry__
from speculative_decode_mla_tree_gb300 import abi
from speculative_decode_mla_tree_gb300.step import DecodeStep

import paged_ref as ref

pytestmark = pytest.mark.gpu
SCALE = 1.0 / math.sqrt(192.0)
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    __graft_entry__.build()


def normal(g, *shape, dtype=BF):
    return torch.randn(*shape, generator=g).to(dtype)


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def paged(g, lens, page, extra=3, gap=0, max_pages=None):
    """(cache [pages, page, 576] on the GPU with page stride page * 576 + gap,
    flat CPU copy, CPU table with garbage behind the used entries): rows in
    use drawn, all others NaN."""
    used = [-(-n // page) for n in lens]
    width = max(used + [1]) + 1 if max_pages is None else max_pages
    pages = sum(used) + extra
    order = torch.randperm(pages, generator=g)
    table = torch.full((len(lens), width), -(1 << 30), dtype=torch.int32)
    table[:, 1::2] = 1 << 30
    flat = torch.full((pages * page, 576), float("nan"), dtype=BF)
    at = 0
    for b, n in enumerate(lens):
        table[b, :used[b]] = order[at:at + used[b]].int()
        at += used[b]
        if n:
            flat[ref.slots_of(table[b], page, 0, n)] = normal(g, n, 576)
    store = torch.full((pages, page * 576 + gap), float("nan"), dtype=BF, device="cuda")
    cache = store[:, :page * 576].unflatten(1, (page, 576))
    cache.copy_(flat.view(pages, page, 576))
    return cache, flat, table


def decode(q, cache, table, lens, status=None, workspace=None, scale=SCALE, fill=7.0):
    B, H, _ = q.shape
    out = torch.full((B, H, 512), fill, dtype=BF, device="cuda")
    lse = torch.full((B, H), fill, device="cuda")
    if workspace is None:
        workspace = torch.full((abi.mla_paged_decode_workspace_bytes(B, H),), 255, dtype=torch.uint8, device="cuda")
    abi.mla_paged_decode(q, cache, table, lens, scale, out, lse, workspace, status)
    return out, lse


def check(out, lse, want, rows=slice(None)):
    wo, wl, to, tl = (x[rows] for x in want)
    o, l = out.double().cpu()[rows], lse.double().cpu()[rows]
    empty = torch.isneginf(wl)
    assert torch.equal(torch.isneginf(l), empty)
    assert (o[empty] == 0).all()
    assert torch.isfinite(o).all()
    assert ((o - wo).abs() <= to).all(), ((o - wo).abs() / to.clamp_min(1e-30)).max()
    off = torch.where(empty, torch.zeros_like(l), (l - wl).abs())
    assert (off <= tl).all(), (off / tl.clamp_min(1e-30)).max()


RAGGED = [0, 1, 2, 63, 64, 65, 127, 128, 129, 191, 300, 1000]


def run_decode(seed, lens, heads, page, gap=0, q=None):
    g = gen(seed)
    cache, flat, table = paged(g, lens, page, gap=gap)
    q = normal(g, len(lens), heads, 576) if q is None else q
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = decode(q.cuda(), cache, table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), status)
    want = ref.decode(q, flat, table, lens, page, SCALE)
    check(out, lse, want)
    assert int(status) == 0
    return out, lse


@pytest.mark.parametrize("page", [8, 16, 32, 64, 128, 256, 24, 40, 48, 72, 1, 3, 20])
def test_decode_pages(page):
    run_decode(page, RAGGED, 16, page)


@pytest.mark.parametrize("heads", [1, 7, 8, 16, 17, 24, 32, 33, 63, 64, 65, 100, 128, 130, 200])
@pytest.mark.parametrize("page,gap", [(64, 0), (5, 0), (5, 8)], ids=["boxes", "rows", "any"])
def test_decode_heads(heads, page, gap):
    run_decode(heads, [1, 100, 0, 513], heads, page, gap)


@pytest.mark.parametrize("page", [1, 3, 20])
def test_decode_any_layout(page):
    """Page strides that are no whole number of rows."""
    run_decode(page, RAGGED, 16, page, gap=40)
    run_decode(page, [5000, 1], 24, page, gap=40)


@pytest.mark.parametrize("batch", [1, 2, 151, 152, 153, 400, 1100])
def test_decode_batches(batch):
    r = torch.randint(0, 130, (batch,), generator=gen(batch)).tolist()
    run_decode(batch, r, 8, 32)


@pytest.mark.parametrize("heads", [8, 64, 128])
def test_decode_one_long_request(heads):
    """Split over the whole card and joined."""
    run_decode(5, [20011], heads, 64)


def test_decode_long_next_to_short():
    run_decode(6, [1, 9000, 0, 3, 12000, 64], 24, 16)


def test_decode_same_in_every_run():
    g = gen(7)
    lens = [3000, 1, 700, 5000]
    cache, _, table = paged(g, lens, 32)
    q, t, n = normal(g, 4, 64, 576).cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    one = decode(q, cache, t, n)
    for _ in range(5):
        two = decode(q, cache, t, n)
        assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])


@pytest.mark.parametrize("page", [64, 16, 3])
def test_decode_strides(page):
    """Queries inside a wider buffer, heads outermost; pages with room between
    them; a table inside a wider one."""
    g = gen(8)
    lens = [130, 64, 1, 777]
    cache, flat, table = paged(g, lens, page, gap=576 * 2)
    q = normal(g, 4, 20, 576)
    wide = torch.full((20, 4, 640), float("nan"), dtype=BF, device="cuda")
    wide[:, :, :576] = q.transpose(0, 1).cuda()
    big = torch.full((4, table.shape[1] + 9), 1 << 30, dtype=torch.int32, device="cuda")
    big[:, :table.shape[1]] = table.cuda()
    out, lse = decode(wide[:, :, :576].transpose(0, 1), cache, big[:, :table.shape[1]],
                      torch.tensor(lens, dtype=torch.int32, device="cuda"))
    check(out, lse, ref.decode(q, flat, table, lens, page, SCALE))


@pytest.mark.parametrize("kind", ["peaked", "equal", "far_below", "huge_values", "growing"])
@pytest.mark.parametrize("page,gap", [(64, 0), (1, 0), (1, 8)], ids=["boxes", "rows", "any"])
def test_decode_scores(kind, page, gap):
    """Softmaxes that rest on one key, on all alike, on scores far below zero,
    values beyond 16-bit range, maxima that rise with every tile."""
    g = gen(9)
    lens = [1000, 65, 3]
    cache, flat, table = paged(g, lens, page, gap=gap)
    q = normal(g, 3, 40, 576)
    if kind == "peaked":
        q = q * 16
    elif kind == "equal":
        q = q * 0
    elif kind == "far_below":
        flat[:, 512:] = torch.where(torch.isnan(flat[:, 512:]), flat[:, 512:], torch.full_like(flat[:, 512:], -8.0))
        q[:, :, 512:] = 8.0
    elif kind == "huge_values":
        flat *= 2.0 ** 60
        q = q * 2.0 ** -60
    else:
        for b, n in enumerate(lens):
            rows = ref.slots_of(table[b], page, 0, n)
            flat[rows, 512:] = (torch.arange(n) / 16.0)[:, None].expand(-1, 64).to(BF)
        q[:, :, 512:] = 1.0
    cache.copy_(flat.view(cache.shape))
    out, lse = decode(q.cuda(), cache, table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"))
    check(out, lse, ref.decode(q, flat, table, lens, page, SCALE))


@pytest.mark.parametrize("page,gap", [(64, 0), (16, 0), (8, 0), (24, 0), (7, 0), (7, 8)])
def test_decode_bad_pages_and_lengths(page, gap):
    """A bad page's positions are left out; a bad length leaves its rows as they were."""
    g = gen(10)
    lens = [500, 200, 70, 64, 90]
    cache, flat, table = paged(g, lens, page, gap=gap)
    pages = cache.shape[0]
    bad = [-1, pages, -(1 << 31), (1 << 31) - 1]
    table[0, 1], table[0, 500 // page - 1] = bad[0], bad[1]
    table[1, 0] = bad[2]
    table[2, : -(-70 // page)] = bad[3]  # nothing is left of this request
    given = list(lens)
    given[3], given[4] = -1, table.shape[1] * page + 1
    q = normal(g, 5, 12, 576)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = decode(q.cuda(), cache, table.cuda(), torch.tensor(given, dtype=torch.int32, device="cuda"), status)
    want = ref.decode(q, flat, table, lens[:3] + [0, 0], page, SCALE, bad_pages=bad)
    check(out, lse, want, slice(0, 3))
    assert (out[3:] == 7.0).all() and (lse[3:] == 7.0).all()
    assert int(status) == abi.DEV_BAD_SLOT | abi.DEV_BAD_INDPTR


def test_decode_far_rows():
    """Pages behind the 2^32nd byte and the 2^31st element of the cache."""
    page, pages = 64, 60000
    cache = torch.empty(pages, page, 576, dtype=BF, device="cuda")
    assert cache.numel() > 2 ** 31
    lens, g = [200, 64], gen(11)
    table = torch.tensor([[pages - 1, 0, pages - 2, 59001], [58999, 0, 0, 0]], dtype=torch.int32)
    flat = torch.zeros(pages * page, 576, dtype=BF)
    for p in table.unique().tolist():
        rows = normal(g, page, 576)
        cache[p] = rows.cuda()
        flat[p * page:(p + 1) * page] = rows
    q = normal(g, 2, 64, 576)
    out, lse = decode(q.cuda(), cache, table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"))
    check(out, lse, ref.decode(q, flat, table, lens, page, SCALE))


def test_decode_captured_with_other_lengths():
    """One captured call replayed on new queries, lengths and tables, and two
    captured calls with workspaces of their own on two streams."""
    g = gen(12)
    B, H, page, width = 5, 64, 32, 80
    cases = []
    for lens in ([2000, 1, 0, 500, 33], [1, 2500, 64, 0, 0], [0] * 5):
        cases.append((lens,) + paged(gen(13), [2560] * B, page, max_pages=width) + (normal(g, B, H, 576),))
    cache = cases[0][1]
    q = torch.zeros(B, H, 576, dtype=BF, device="cuda")
    table = torch.zeros(B, width, dtype=torch.int32, device="cuda")
    n = torch.zeros(B, dtype=torch.int32, device="cuda")
    outs = [(torch.zeros(B, H, 512, dtype=BF, device="cuda"), torch.zeros(B, H, device="cuda")) for _ in range(2)]
    ws = [torch.zeros(abi.mla_paged_decode_workspace_bytes(B, H), dtype=torch.uint8, device="cuda") for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    graphs = []
    for k in range(2):
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=streams[k]):
            abi.mla_paged_decode(q, cache, table, n, SCALE, *outs[k], ws[k])
        graphs.append(graph)
    for lens, _, flat, tab, queries in cases:
        q.copy_(queries)
        table.copy_(tab)
        n.copy_(torch.tensor(lens))
        torch.cuda.synchronize()
        for _ in range(3):
            for graph, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    graph.replay()
        torch.cuda.synchronize()
        want = ref.decode(queries, flat, tab, lens, page, SCALE)
        for o, l in outs:
            check(o, l, want)


@pytest.mark.parametrize("heads", [8, 64, 128])
@pytest.mark.parametrize("drop", [0, 3])
@pytest.mark.parametrize("page", [32, 3])
def test_decode_wait_gives_up_then_next_call_is_correct(heads, drop, page):
    """With its copies withheld from one share on, the tensor-core kernel
    reports the timeout and leaves the device usable; the next call is right."""
    g = gen(14)
    lens = [1500, 900, 64, 2000]
    cache, flat, table = paged(g, lens, page)
    q = normal(g, 4, heads, 576)
    args = (q.cuda(), cache, table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    decode(*args, status)
    assert int(status) == 0
    abi.mla_tree_test_wait_limits(drop, 1_000_000)
    try:
        decode(*args, status)
        torch.cuda.synchronize()
    finally:
        abi.mla_tree_test_wait_limits(-1, 0)
    assert int(status) == abi.DEV_TIMEOUT
    status.zero_()
    out, lse = decode(*args, status)
    check(out, lse, ref.decode(q, flat, table, lens, page, SCALE))
    assert int(status) == 0


@pytest.mark.parametrize("page,gap", [(64, 0), (6, 0), (6, 8)])
def test_decode_not_a_number(page, gap):
    """A NaN in a visible key row makes the heads of that request NaN, and no other's."""
    g = gen(15)
    lens = [700, 700, 5]
    cache, flat, table = paged(g, lens, page, gap=gap)
    flat[ref.slots_of(table[1], page, 300, 301), 3] = float("nan")
    cache.copy_(flat.view(cache.shape))
    q = normal(g, 3, 16, 576)
    out, lse = decode(q.cuda(), cache, table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"))
    assert torch.isnan(lse[1]).all() and torch.isnan(out[1]).all()
    want = ref.decode(q, flat, table, [700, 0, 5], page, SCALE)
    for b in (0, 2):
        check(out, lse, want, slice(b, b + 1))


# ------------------------------------------------------------------- append

def rope_table(n, base=10000.0):
    f = base ** (-torch.arange(32, dtype=torch.float64) / 32)
    a = torch.arange(n, dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def run_append(seed, new, lens, page, heads, halves=False, norm=False, depths=False, in_place=False, gap=0, pad=0,
               table_hook=None):
    """Appends and compares everything: the rows written, the rest untouched."""
    g = gen(seed)
    T = sum(new) + pad
    cache, flat, table = paged(g, lens, page, gap=gap)
    if table_hook:
        table_hook(table, cache.shape[0])
    row, proj = normal(g, T, 576 + 64), normal(g, T, max(heads, 1), 192)
    weight = normal(g, 512) if norm else None
    indptr = torch.tensor([0] + new).cumsum(0).int()
    n = torch.tensor(lens, dtype=torch.int32)
    table_rope = rope_table(max(lens) + 50)
    pos = torch.randint(0, max(lens) + 50, (T,), generator=g).int() if depths else None
    latent, k_rope, q_rope = row[:, :512], row[:, 512:576], proj[:, :heads, 128:]
    grow, gproj = row.cuda(), proj.cuda()
    qin = gproj[:, :heads, 128:]
    qbuf = torch.full((T, max(heads, 1), 576), 5.0, dtype=BF, device="cuda")
    qout = qin if in_place else qbuf[:, :heads, 512:]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    before = cache.clone()
    abi.mla_paged_append(grow[:, :512], grow[:, 512:576], indptr.cuda(), n.cuda(), table.cuda(), cache,
                         table_rope.cuda(), qin if heads else None, qout if heads else None,
                         None if pos is None else pos.cuda(), None if weight is None else weight.cuda(), 1e-6,
                         abi.ROPE_HALVES if halves else abi.ROPE_PAIRS, status)
    slots, rows, rtol, qs, qtol = ref.append(latent, k_rope, indptr, n, table, flat, page, table_rope,
                                             q_rope if heads else None, pos, weight, 1e-6, halves)
    got = cache.cpu().reshape(-1, 576)
    assert ((got[slots].double() - rows).abs() <= rtol).all()
    if not norm:
        assert torch.equal(got[slots][:, :512], latent[: sum(new)])
    keep = torch.ones(got.shape[0], dtype=torch.bool)
    keep[slots] = False
    assert torch.equal(got[keep].view(torch.int16), before.cpu().reshape(-1, 576)[keep].view(torch.int16))
    if heads:
        q = qout.cpu()
        assert ((q[: sum(new)].double() - qs).abs() <= qtol).all()
        untouched = proj[sum(new):, :heads, 128:] if in_place else torch.full_like(q[sum(new):], 5.0)
        assert torch.equal(q[sum(new):], untouched)
        if in_place:
            assert torch.equal(gproj[:, :, :128].cpu(), proj[:, :, :128])
        else:
            assert (qbuf[:, :, :512] == 5.0).all()
    assert int(status) == 0


@pytest.mark.parametrize("halves", [False, True], ids=["pairs", "halves"])
@pytest.mark.parametrize("norm", [False, True], ids=["copy", "norm"])
@pytest.mark.parametrize("heads", [0, 1, 3, 8, 16, 17, 64, 128])
def test_append_forms(halves, norm, heads):
    run_append(heads, [3, 0, 1, 70, 0], [3, 0, 40, 100, 7], 16, heads, halves, norm)


@pytest.mark.parametrize("page", [1, 3, 16, 64, 256])
def test_append_pages(page):
    run_append(page, [1, 5, 300, 0, 64], [1, 90, 301, 0, 64], page, 5, norm=True, gap=576)


@pytest.mark.parametrize("batch", [1, 31, 32, 33, 1000, 1025])
def test_append_batches(batch):
    new = torch.randint(0, 3, (batch,), generator=gen(batch)).tolist()
    past = torch.randint(0, 50, (batch,), generator=gen(batch + 1)).tolist()
    run_append(batch, new, [a + b for a, b in zip(new, past)], 16, 2, depths=True)


@pytest.mark.parametrize("halves", [False, True], ids=["pairs", "halves"])
def test_append_in_place_and_padded(halves):
    """Queries rotated where they are; tokens behind the last request left alone."""
    run_append(3, [7, 1, 9], [7, 30, 33], 32, 20, halves, in_place=True, pad=5)
    run_append(4, [7, 1, 9], [7, 30, 33], 32, 20, halves, pad=5)


def test_append_far_positions():
    """Angles of a position beyond 2^20 come from the table as they are."""
    g = gen(20)
    n, page = 1 << 20, 64
    table_rope = rope_table(n + 1)
    cache = torch.zeros(2, page, 576, dtype=BF, device="cuda")
    row = normal(g, 2, 576)
    pos = torch.tensor([n, n - 1], dtype=torch.int32)
    abi.mla_paged_append(row[:, :512].cuda(), row[:, 512:].cuda(), torch.tensor([0, 2], dtype=torch.int32).cuda(),
                         torch.tensor([2], dtype=torch.int32).cuda(), torch.tensor([[1]], dtype=torch.int32).cuda(),
                         cache, table_rope.cuda(), positions=pos.cuda())
    _, rows, tol, _, _ = ref.append(row[:, :512], row[:, 512:], [0, 2], [2], [[1]], None, page, table_rope,
                                    positions=pos)
    assert ((cache[1, :2].double().cpu() - rows).abs() <= tol).all()


def _bad_append(indptr, lens, table, positions=None, max_positions=60, T=6):
    g = gen(30)
    cache = torch.full((4, 16, 576), 3.0, dtype=BF, device="cuda")
    row, q = normal(g, T, 576).cuda(), normal(g, T, 4, 64).cuda()
    qout = torch.full_like(q, 5.0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    abi.mla_paged_append(row[:, :512], row[:, 512:], i32(indptr), i32(lens), i32(table), cache,
                         rope_table(max_positions).cuda(), q, qout, None if positions is None else i32(positions),
                         status=status)
    rows = (cache != 3.0).any(-1).nonzero().tolist()
    return int(status), rows, (qout != 5.0).flatten(1).any(1).tolist()


def test_append_bad_contents():
    """Each bad value sets its bit and leaves out what it names, nothing else."""
    first = [[0, 0], [0, 1], [0, 2]]
    ok = (0, first + [[1, 3], [1, 4], [1, 5]], [True] * 6)
    assert _bad_append([0, 3, 6], [3, 6], [[0], [1]]) == ok
    for page in (-1, 4, 1 << 30):
        assert _bad_append([0, 3, 6], [3, 6], [[0], [page]]) == (abi.DEV_BAD_SLOT, first, [True] * 6)
    for n in (2, -1, 17):  # shorter than its new tokens, negative, beyond the table
        assert _bad_append([0, 3, 6], [3, n], [[0], [1]]) == (abi.DEV_BAD_INDPTR, first, [True] * 3 + [False] * 3)
    assert _bad_append([0, 3, 9], [3, 9], [[0], [1]]) == (abi.DEV_BAD_INDPTR, first, [True] * 3 + [False] * 3)
    for p in (-1, 60):
        assert _bad_append([0, 3, 6], [3, 6], [[0], [1]], [0, 1, 2, 3, p, 5]) == (
            abi.DEV_BAD_POSITION, first + [[1, 3], [1, 5]], [True] * 4 + [False, True])
    status, rows, _ = _bad_append([0, 7, 6], [7, 6], [[0], [1]])
    assert status & abi.DEV_BAD_INDPTR and not [r for r in rows if r[0] > 1]
    status, _, _ = _bad_append([5, 3, 6], [3, 6], [[0], [1]])
    assert status & abi.DEV_BAD_INDPTR


# ------------------------------------------------------------- used together

@pytest.mark.parametrize("heads", [8, 64])
def test_prompt_then_decode_then_tree(heads):
    """A cache filled with prompts in two chunks, a decoding step captured and
    replayed token by token, then a draft tree appended at its depths and
    verified through the same cache seen as a slot pool."""
    g = gen(40 + heads)
    page, lens = 16, [37, 150, 5]
    B, width, steps = 3, 12, 4
    rope = rope_table(256)
    cache = torch.full((B * width, page, 576), float("nan"), dtype=BF, device="cuda")
    table = torch.randperm(B * width, generator=g).int().view(B, width)
    flat = torch.zeros(B * width * page, 576, dtype=BF)
    weight = normal(g, 512)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731

    def mirror(slots, rows, tol):
        got = cache.cpu().reshape(-1, 576)[slots]
        assert ((got.double() - rows).abs() <= tol).all()
        flat[slots] = got

    done = [0] * B
    for part in ([20, 150, 0], [17, 0, 5]):
        done = [a + b for a, b in zip(done, part)]
        T = sum(part)
        row = normal(g, T, 576)
        ptr = [0] + torch.tensor(part).cumsum(0).tolist()
        abi.mla_paged_append(row[:, :512].cuda(), row[:, 512:].cuda(), i32(ptr), i32(done), table.cuda(), cache,
                             rope.cuda(), norm_weight=weight.cuda())
        mirror(*ref.append(row[:, :512], row[:, 512:], ptr, done, table, None, page, rope, weight=weight)[:3])
    assert done == lens

    step = DecodeStep(cache, B, heads, width, rope.cuda(), SCALE, norm_weight=weight.cuda())
    step.block_table.copy_(table)
    step.kv_lens.copy_(i32(lens) + 1)
    step.latent.copy_(normal(g, B, 512))
    step.run()  # warm-up outside the graph; the first replayed step writes the same rows again
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.run()
    for k in range(steps):
        now = [n + k + 1 for n in lens]
        row, q = normal(g, B, 576), normal(g, B, heads, 576)
        step.kv_lens.copy_(i32(now))
        step.latent.copy_(row[:, :512])
        step.k_rope.copy_(row[:, 512:])
        step.q.copy_(q)
        graph.replay()
        torch.cuda.synchronize()
        slots, rows, tol, qs, qtol = ref.append(row[:, :512], row[:, 512:], list(range(B + 1)), now, table, None, page,
                                                rope, q[:, :, 512:], weight=weight)
        mirror(slots, rows, tol)
        turned = step.q.cpu()
        assert torch.equal(turned[:, :, :512], q[:, :, :512])
        assert ((turned[:, :, 512:].double() - qs).abs() <= qtol).all()
        check(step.out, step.lse, ref.decode(turned, flat, table, now, page, SCALE))
    assert int(step.status) == 0

    # a draft tree of 4 nodes a request: 0 -> 1, 0 -> 2, 2 -> 3
    past = [n + steps for n in lens]
    full = [p + 4 for p in past]
    depth = torch.tensor([[p, p + 1, p + 1, p + 2] for p in past]).int().flatten()
    row, q = normal(g, 12, 576), normal(g, 12, heads, 576).cuda()
    ptr = [0, 4, 8, 12]
    abi.mla_paged_append(row[:, :512].cuda(), row[:, 512:].cuda(), i32(ptr), i32(full), table.cuda(), cache,
                         rope.cuda(), q[:, :, 512:], q[:, :, 512:], depth.cuda(), weight.cuda())
    mirror(*ref.append(row[:, :512], row[:, 512:], ptr, full, table, None, page, rope, positions=depth,
                       weight=weight)[:3])
    slots = [ref.slots_of(table[b], page, 0, full[b]).int() for b in range(B)]
    kv_indices = torch.cat(slots).cuda()
    kv_ptr = i32([0] + torch.tensor(full).cumsum(0).tolist())
    words = torch.zeros(sum(4 * ((n + 31) // 32) for n in full), dtype=torch.int32, device="cuda")
    wptr = torch.zeros(B + 1, dtype=torch.int64, device="cuda")
    abi.tree_mask_pack_bits(i32([-1, 0, 0, 2] * B), i32(ptr), kv_ptr, wptr, words)
    out = torch.zeros(12, heads, 512, dtype=BF, device="cuda")
    lse = torch.zeros(12, heads, device="cuda")
    ws = torch.empty(max(256, abi.mla_tree_verify_workspace_bytes(B, 12, heads)), dtype=torch.uint8, device="cuda")
    abi.mla_tree_verify_bits(q, cache.view(-1, 576), kv_indices, kv_ptr, i32(ptr), words, wptr, SCALE, out, lse, ws)
    sees = [[0], [0, 1], [0, 2], [0, 2, 3]]
    for b in range(B):
        for node in range(4):
            keep = torch.cat([slots[b][:past[b]], slots[b][past[b] + torch.tensor(sees[node])]]).long()
            own = [keep.tolist()]
            want = ref.decode(q[4 * b + node].cpu()[None], flat, own, [len(own[0])], 1, SCALE)
            check(out[4 * b + node][None], lse[4 * b + node][None], want)


# ----------------------------------------------------------------- refusals

def _decode_args():
    g = gen(50)
    cache, _, table = paged(g, [100, 20], 32)
    return dict(q=normal(g, 2, 8, 576).cuda(), cache=cache, block_table=table.cuda(),
                kv_lens=torch.tensor([100, 20], dtype=torch.int32, device="cuda"), sm_scale=SCALE,
                out=torch.full((2, 8, 512), 7.0, dtype=BF, device="cuda"), lse=torch.full((2, 8), 7.0, device="cuda"),
                workspace=torch.empty(abi.mla_paged_decode_workspace_bytes(2, 8), dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("name,change", [
    ("q", lambda t: t.float()), ("q", lambda t: t.cpu()), ("q", lambda t: t[:, :, :575]), ("q", lambda t: t[:1]),
    ("q", lambda t: None), ("q", lambda t: t.permute(0, 2, 1)), ("q", lambda t: t[0]),
    ("q", lambda t: t[:, :1].expand(2, 8, 576)),
    ("cache", lambda t: t.half()), ("cache", lambda t: t.cpu()), ("cache", lambda t: t[:, :, :512]),
    ("cache", lambda t: t.flatten(0, 1)), ("cache", lambda t: t[:, ::2]), ("cache", lambda t: 5),
    ("block_table", lambda t: t.long()), ("block_table", lambda t: t.cpu()), ("block_table", lambda t: t[:, ::2]),
    ("block_table", lambda t: t[:1]), ("block_table", lambda t: t.flatten()),
    ("kv_lens", lambda t: t.long()), ("kv_lens", lambda t: t[:1]), ("kv_lens", lambda t: [100, 20]),
    ("out", lambda t: t.float()), ("out", lambda t: t[:, :4]), ("out", lambda t: t.transpose(0, 1).contiguous().transpose(0, 1)),
    ("lse", lambda t: t.half()), ("lse", lambda t: t[:, :4]), ("workspace", lambda t: t[:-1]),
    ("workspace", lambda t: t[1:]), ("workspace", lambda t: t.int()), ("workspace", lambda t: None),
    ("sm_scale", lambda t: float("nan"))])
def test_decode_refuses(name, change):
    """What does not fit is refused before anything is launched."""
    args = _decode_args()
    out, lse = args["out"], args["lse"]
    args[name] = change(args[name])
    with pytest.raises(abi.MlaTreeError):
        abi.mla_paged_decode(**args)
    torch.cuda.synchronize()
    assert (out == 7.0).all() and (lse == 7.0).all()


def _append_args():
    g = gen(51)
    cache = torch.full((4, 16, 576), 3.0, dtype=BF, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    row = normal(g, 6, 576).cuda()
    return dict(latent=row[:, :512], k_rope=row[:, 512:], qo_indptr=i32([0, 3, 6]), kv_lens=i32([3, 6]),
                block_table=i32([[0], [1]]), cache=cache, rope_table=rope_table(64).cuda(),
                q_rope=normal(g, 6, 4, 64).cuda(), q_out=torch.full((6, 4, 64), 5.0, dtype=BF, device="cuda"),
                positions=i32([0, 1, 2, 3, 4, 5]), norm_weight=normal(g, 512).cuda())


@pytest.mark.parametrize("name,change", [
    ("latent", lambda t: t.float()), ("latent", lambda t: t[:, :511]), ("latent", lambda t: t[:5]),
    ("latent", lambda t: t.cpu()), ("latent", lambda t: None), ("k_rope", lambda t: t[:, :63]),
    ("k_rope", lambda t: t[:5]), ("qo_indptr", lambda t: t[:2]), ("qo_indptr", lambda t: t.long()),
    ("kv_lens", lambda t: t.repeat(2)[::2]), ("block_table", lambda t: t.float()), ("cache", lambda t: t.float()),
    ("rope_table", lambda t: t.double()), ("rope_table", lambda t: t[:, :32]), ("rope_table", lambda t: t.t()),
    ("q_rope", lambda t: None), ("q_out", lambda t: None), ("q_out", lambda t: t[:, :3]),
    ("q_out", lambda t: t.float()), ("q_rope", lambda t: t[:, :, :32]), ("q_out", lambda t: t[:1].expand(6, 4, 64)),
    ("positions", lambda t: t.long()), ("positions", lambda t: t[:5]), ("norm_weight", lambda t: t.float()),
    ("norm_weight", lambda t: t[:511]), ("rope_style", lambda t: 2), ("norm_eps", lambda t: -1.0)])
def test_append_refuses(name, change):
    args = _append_args()
    cache, q_out = args["cache"], args["q_out"]
    args[name] = change(args.get(name))
    with pytest.raises(abi.MlaTreeError):
        abi.mla_paged_append(**args)
    torch.cuda.synchronize()
    assert (cache == 3.0).all() and (q_out == 5.0).all()
