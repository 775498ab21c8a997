"""Window decode on the GPU against its formula in 64 bits: the visible
positions of a request are gathered into a table of slots (page size 1), whose
plain attention paged_ref states with its bounds. Rows that no visible position
has hold NaN, and table entries of pages without any are garbage."""
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


def visible(n, window, sinks):
    return [j for j in range(n) if j < sinks or j >= n - window]


def windowed(g, lens, page, window, sinks, gap=0):
    """(cache on the GPU, flat CPU copy, table, table of the visible slots, their numbers)"""
    seen = [visible(n, window, sinks) for n in lens]
    cols = [sorted({j // page for j in s}) for s in seen]
    width = max([-(-n // page) for n in lens] + [1]) + 1
    pages = sum(len(c) for c in cols) + 3
    order = torch.randperm(pages, generator=g).tolist()
    table = torch.full((len(lens), width), -(1 << 30), dtype=torch.int32)
    table[:, 1::2] = 1 << 30
    flat = torch.full((pages * page, 576), float("nan"), dtype=BF)
    slots = torch.zeros(len(lens), max([len(s) for s in seen] + [1]), dtype=torch.int32)
    at = 0
    for b, s in enumerate(seen):
        for c in cols[b]:
            table[b, c] = order[at]
            at += 1
        if s:
            ids = torch.tensor([int(table[b, j // page]) * page + j % page for j in s])
            flat[ids] = torch.randn(len(s), 576, generator=g).to(BF)
            slots[b, :len(s)] = ids.int()
    store = torch.full((pages, page * 576 + gap), float("nan"), dtype=BF, device="cuda")
    cache = store[:, :page * 576].unflatten(1, (page, 576))
    cache.copy_(flat.view(pages, page, 576))
    return cache, flat, table, slots, [len(s) for s in seen]


def decode(q, cache, table, lens, window, sinks, status=None, stream=None):
    B, H, _ = q.shape
    out = torch.full((B, H, 512), 7.0, dtype=BF, device="cuda")
    lse = torch.full((B, H), 7.0, device="cuda")
    ws = torch.full((abi.mla_paged_decode_workspace_bytes(B, H),), 255, dtype=torch.uint8, device="cuda")
    abi.mla_paged_decode_window(q, cache, table, lens, window, sinks, SCALE, out, lse, ws, status, stream)
    return out, lse


def check(out, lse, want):
    wo, wl, to, tl = want
    o, l = out.double().cpu(), lse.double().cpu()
    empty = torch.isneginf(wl)
    assert torch.equal(torch.isneginf(l), empty) and (o[empty] == 0).all() and torch.isfinite(o).all()
    assert ((o - wo).abs() <= to).all(), ((o - wo).abs() / to.clamp_min(1e-30)).max()
    off = torch.where(empty, torch.zeros_like(l), (l - wl).abs())
    assert (off <= tl).all(), (off / tl.clamp_min(1e-30)).max()


def run(seed, lens, heads, page, window, sinks, gap=0):
    g = torch.Generator()
    g.manual_seed(seed)
    cache, flat, table, slots, counts = windowed(g, lens, page, window, sinks, gap)
    q = torch.randn(len(lens), heads, 576, generator=g).to(BF)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = decode(q.cuda(), cache, table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), window, sinks,
                      status)
    check(out, lse, ref.decode(q, flat, slots, counts, 1, SCALE))
    assert int(status) == 0
    return out, lse


def around(window, sinks):
    """Lengths where the edges of the window, the sinks and the units of 8 and 16 rows meet."""
    e = window + sinks
    return sorted({0, 1, 2, 63, 65, 300, 1000, *(max(0, e + d) for d in (-1, 0, 1, 7, 8, 9, 15, 16, 17, 33, 64, 100))})


SHAPES = [(1, 0), (1, 1), (1, 5), (7, 0), (16, 16), (17, 3), (64, 4), (100, 64), (130, 130), (512, 1), (10, 700), (2000, 5)]


@pytest.mark.parametrize("page,gap", [(8, 0), (16, 0), (64, 0), (24, 0), (40, 0), (128, 0), (1, 0), (5, 0), (20, 0), (5, 8), (1, 40)])
@pytest.mark.parametrize("window,sinks", SHAPES)
def test_edges(page, gap, window, sinks):
    run(window + page, around(window, sinks), 8, page, window, sinks, gap)


@pytest.mark.parametrize("heads", [1, 16, 17, 33, 64, 65, 128, 130])
@pytest.mark.parametrize("page,gap", [(64, 0), (3, 0), (3, 8)], ids=["boxes", "rows", "any"])
def test_heads(heads, page, gap):
    run(heads, [1, 700, 0, 260, 5000], heads, page, 201, 9, gap)


@pytest.mark.parametrize("batch", [1, 2, 151, 153, 400])
def test_batches(batch):
    g = torch.Generator()
    g.manual_seed(batch)
    run(batch, torch.randint(0, 900, (batch,), generator=g).tolist(), 8, 32, 100, 20)


@pytest.mark.parametrize("heads", [8, 24, 64, 128])
@pytest.mark.parametrize("batch,window,sinks", [(1, 500, 4), (9, 500, 4), (14, 100, 0), (30, 100, 0), (60, 60, 3), (3, 1500, 0)])
@pytest.mark.parametrize("page", [16, 9])
def test_one_cluster_a_request(heads, batch, window, sinks, page):
    """Requests of no tile, one, fewer than the cluster has CTAs, and more."""
    g = torch.Generator()
    g.manual_seed(batch)
    lens = torch.randint(0, window + 300, (batch,), generator=g).tolist()
    lens[0] = window + 250
    lens[-1] = 5
    lens[batch // 2] = 0
    run(batch + heads, lens, heads, page, window, sinks)


def test_same_in_every_run():
    for heads, window in ((8, 400), (64, 100), (64, 3000)):
        a = run(1, [5000, 90, 700, 0], heads, 64, window, 4)
        b = run(1, [5000, 90, 700, 0], heads, 64, window, 4)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_timeout_in_a_cluster():
    """A wait that runs out is said; nothing is written for that request, and the next call is right."""
    g = torch.Generator()
    g.manual_seed(5)
    cache, flat, table, slots, counts = windowed(g, [900, 900], 64, 500, 4)
    q = torch.randn(2, 8, 576, generator=g).to(BF)
    n = torch.tensor([900, 900], dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    abi.mla_tree_test_wait_limits(9, 50_000_000)  # of the second request's eight parts, all but the first
    try:
        out, lse = decode(q.cuda(), cache, table.cuda(), n, 500, 4, status)
        assert int(status) == abi.DEV_TIMEOUT
    finally:
        abi.mla_tree_test_wait_limits(-1, 0)
    want = ref.decode(q, flat, slots, counts, 1, SCALE)
    check(out[:1], lse[:1], tuple(w[:1] for w in want))
    assert (out[1] == 7).all() and (lse[1] == 7).all()
    status.zero_()
    out, lse = decode(q.cuda(), cache, table.cuda(), n, 500, 4, status)
    check(out, lse, want)
    assert int(status) == 0


@pytest.mark.parametrize("page", [64, 16, 7])
def test_long_window_is_split(page):
    run(page, [40000, 12345], 16, page, 9000, 70)


@pytest.mark.parametrize("heads,page", [(8, 64), (64, 16), (16, 5)])
@pytest.mark.parametrize("window,sinks", [(1 << 20, 0), ((1 << 31) - 1, (1 << 31) - 1), (1, (1 << 31) - 1), (1001, 0), (1, 1000)])
def test_all_visible_is_the_plain_call(heads, page, window, sinks):
    """Bit for bit where the table holds no more; else within the rounding of other splits."""
    g = torch.Generator()
    g.manual_seed(heads)
    lens = [0, 1, 500, 1001]
    cache, flat, table, slots, counts = windowed(g, lens, page, 1 << 20, 0)
    q = torch.randn(4, heads, 576, generator=g).to(BF)
    t, n = table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    out, lse = decode(q.cuda(), cache, t, n, window, sinks)
    check(out, lse, ref.decode(q, flat, slots, counts, 1, SCALE))
    if max(window, sinks) < table.shape[1] * page:
        return
    ws = torch.zeros(abi.mla_paged_decode_workspace_bytes(4, heads), dtype=torch.uint8, device="cuda")
    out2, lse2 = torch.empty_like(out), torch.empty_like(lse)
    abi.mla_paged_decode(q.cuda(), cache, t, n, SCALE, out2, lse2, ws)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


def test_bad_pages_and_lengths():
    """A bad page in the window is left out and said, one in the gap is not looked at; a bad length leaves its rows."""
    g = torch.Generator()
    g.manual_seed(3)
    lens, page, window, sinks = [500, 500, 500], 16, 100, 20
    cache, flat, table, slots, counts = windowed(g, lens, page, window, sinks)
    q = torch.randn(3, 16, 576, generator=g).to(BF)
    table[1, 28] = cache.shape[0]           # positions 448 .. 463, all in the window
    bad = [j for j in visible(500, window, sinks) if j // 16 != 28]
    slots[1, :len(bad)] = torch.tensor([int(table[1, j // 16]) * 16 + j % 16 for j in bad]).int()
    counts[1] = len(bad)
    n = torch.tensor(lens, dtype=torch.int32)
    n[2] = table.shape[1] * page + 1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = decode(q.cuda(), cache, table.cuda(), n.cuda(), window, sinks, status)
    want = ref.decode(q[:2], flat, slots[:2], counts[:2], 1, SCALE)
    check(out[:2], lse[:2], want)
    assert (out[2] == 7).all() and (lse[2] == 7).all()
    assert int(status) == abi.DEV_BAD_SLOT | abi.DEV_BAD_INDPTR


def test_far_positions():
    """Positions near 2^31 - 1: only the window's and the sinks' pages exist."""
    page, window, sinks = 128, 300, 10
    width = ((1 << 31) - 1) // page
    n = width * page - 5
    table = torch.full((1, width), -1, dtype=torch.int32, device="cuda")
    first = (n - window) // page
    cols = [0] + list(range(first, width))
    g = torch.Generator()
    g.manual_seed(8)
    flat = torch.randn(len(cols) * page, 576, generator=g).to(BF)
    for i, c in enumerate(cols):
        table[0, c] = i
    seen = list(range(sinks)) + list(range(n - window, n))
    slots = torch.tensor([[cols.index(j // page) * page + j % page for j in seen]], dtype=torch.int32)
    q = torch.randn(1, 8, 576, generator=g).to(BF)
    out, lse = decode(q.cuda(), flat.view(-1, page, 576).cuda(), table, torch.tensor([n], dtype=torch.int32, device="cuda"),
                      window, sinks)
    check(out, lse, ref.decode(q, flat, slots, [len(seen)], 1, SCALE))


def test_step_with_a_window_in_a_graph():
    """Decoding steps over a sliding window, captured once: appends move on, the window with them."""
    page, window, sinks, n0 = 16, 40, 4, 70
    g = torch.Generator()
    g.manual_seed(11)
    cache = torch.randn(20, page, 576, generator=g).to(BF).cuda()
    rope = torch.cat([torch.ones(128, 32), torch.zeros(128, 32)], 1).cuda()
    step = DecodeStep(cache, 2, 8, 8, rope, SCALE, window=window, sinks=sinks)
    step.block_table.copy_(torch.randperm(20, generator=g)[:16].view(2, 8).int())
    lens = torch.tensor([n0, 0], dtype=torch.int32)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        step.kv_lens.copy_(torch.tensor([n0, 0], dtype=torch.int32))
        step.run()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step.run()
    torch.cuda.synchronize()
    for i in range(5):
        lens[0] += 1
        step.kv_lens.copy_(lens)
        step.latent.copy_(torch.randn(2, 512, generator=g))
        step.k_rope.copy_(torch.randn(2, 64, generator=g))
        q = torch.randn(2, 8, 576, generator=g).to(BF)
        step.q.copy_(q)
        graph.replay()
        torch.cuda.synchronize()
        table = step.block_table.cpu()
        flat = cache.cpu().view(-1, 576)
        seen = visible(int(lens[0]), window, sinks)
        slots = torch.zeros(2, len(seen), dtype=torch.int32)
        slots[0] = torch.tensor([int(table[0, j // page]) * page + j % page for j in seen]).int()
        check(step.out, step.lse, ref.decode(q, flat, slots, [len(seen), 0], 1, SCALE))
    assert int(step.status) == 0
