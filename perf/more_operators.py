"""Cases of the operators around the attention of a latent-attention serving
step.

* logprobs: from the rows of logits, the log probabilities of given tokens,
  the rows' entropies and their most likely tokens.
* window: attention of one new token per request over the paged cache, to the
  last ``window`` positions and the first ``sinks``.
* finish: what ends a verify step. The draft tree is walked along the tokens
  that the model chose, and the accepted nodes' cache rows move up to follow
  the prefix, in every layer.
* beams: branches of generations take the places of others (their pages
  shared), get room for one more token in pages of their own, and what they
  shared of their last page is copied, in every layer.
* copy: whole pages copied to others, in every layer.

``run`` computes them in plain torch operations, or, where ``own`` is set, by
the library's entry points. A cache row is 576 bf16 values; a page holds
``page`` rows; ``table[b, j]`` is the page of request b's positions
``j * page ..``, and ``refs[p]`` says how many table entries hold page p.
"""
import math
import random

import torch

own = False

D_LAT, D_ROW = 512, 576
SM_SCALE = 1.0 / math.sqrt(192.0)
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one generated token, its best alternative alone: latency counts
        {"name": "logprobs_one_token", "op": "logprobs", "rows": 1, "vocab": 32768, "type": "bf16", "given": 1,
         "top": 1, "pad": 0, "masked": 0.0},
        # the rows of 8 draft trees of 16 nodes
        {"name": "logprobs_draft_trees", "op": "logprobs", "rows": 128, "vocab": 131072, "type": "bf16", "given": 1,
         "top": 8, "pad": 0, "masked": 0.0},
        # a generation batch in fp32 behind a grammar that masks most tokens; an odd vocabulary in padded rows
        {"name": "logprobs_constrained", "op": "logprobs", "rows": 256, "vocab": 100003, "type": "fp32", "given": 3,
         "top": 20, "pad": 29, "masked": 0.7},
        # 32 draft trees of 64 nodes
        {"name": "logprobs_many_rows", "op": "logprobs", "rows": 2048, "vocab": 131072, "type": "bf16", "given": 1,
         "top": 5, "pad": 0, "masked": 0.0},
        # a few chats on a shard of 8 heads, a short window
        {"name": "window_small_batch", "op": "window", "batch": 8, "len_min": 1024, "len_max": 4096, "heads": 8,
         "page": 64, "window": 512, "sinks": 4},
        # the 64-request serving mix, lengths 128 to 131072, behind a window of 4096
        {"name": "window_mix", "op": "window", "batch": 64, "len_min": 128, "len_max": 131072, "heads": 64, "page": 64,
         "window": 4096, "sinks": 64},
        # all 128 heads, a window and sinks that end inside small pages
        {"name": "window_all_heads", "op": "window", "batch": 48, "len_min": 2000, "len_max": 16384, "heads": 128,
         "page": 16, "window": 2047, "sinks": 5},
        # one sequence, a 9-node tree: latency alone
        {"name": "finish_one_tree", "op": "finish", "batch": 1, "nodes_min": 9, "nodes_max": 9, "len_max": 30, "page": 64,
         "layers": 1, "accept": 8, "hit": 0.7},
        # the 64-request batch of 8 to 64 nodes, all layers of a model in one cache
        {"name": "finish_batch", "op": "finish", "batch": 64, "nodes_min": 8, "nodes_max": 64, "len_max": 1500, "page": 64,
         "layers": 32, "accept": 16, "hit": 0.8},
        # 8 searches of 4 beams, small pages
        {"name": "beams_small", "op": "beams", "groups": 8, "fan": 4, "len_min": 100, "len_max": 2000, "page": 16,
         "layers": 4, "window": 0, "sinks": 0},
        # 32 prompts sampled 8 times, all behind a window
        {"name": "beams_many", "op": "beams", "groups": 32, "fan": 8, "len_min": 1000, "len_max": 6000, "page": 64,
         "layers": 8, "window": 2048, "sinks": 64},
        # a prefix of 300 pages taken over, eight layers
        {"name": "copy_prefix", "op": "copy", "pages": 300, "page": 64, "layers": 8},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    kind = rng.choice(["logprobs", "logprobs", "window", "window", "finish", "beams", "copy"])
    page = rng.choice([8, 16, 32, 64, 128])
    if kind == "logprobs":
        vocab = rng.choice([_log_int(rng, 200, 262144), _log_int(rng, 20000, 200000), 65536])
        kinds = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        rows = _log_int(rng, 1, min(8192, 268000000 // (vocab * (2 if kinds == "fp32" else 1))))
        return {"op": "logprobs", "rows": rows, "vocab": vocab, "type": kinds, "given": rng.choice([1, 1, 2, 5]),
                "top": rng.choice([1, 2, 5, 8, 20, 32]), "pad": rng.choice([0, 0, 1, 64]),
                "masked": rng.choice([0.0, 0.0, 0.5, 0.99])}
    if kind == "window":
        batch = _log_int(rng, 1, 128)
        window = min(_log_int(rng, 1, 8192), 400000 // batch)
        n = _log_int(rng, max(1, window // 2), max(window, 1600000 // max(batch, 12)))
        return {"op": "window", "batch": batch, "len_min": rng.choice([0, n // 7, n]), "len_max": n,
                "heads": rng.choice([_log_int(rng, 1, 128), rng.choice([8, 16, 32, 64, 128])]), "page": page,
                "window": window, "sinks": rng.choice([0, 1, 4, 16, 100])}
    if kind == "finish":
        batch = _log_int(rng, 1, 128)
        nodes = _log_int(rng, 2, 64)
        return {"op": "finish", "batch": batch, "nodes_min": max(1, nodes // rng.choice([1, 2, 5])), "nodes_max": nodes,
                "len_max": _log_int(rng, 64, 800), "page": page, "layers": _log_int(rng, 1, max(1, 1500 // batch // 4)),
                "accept": _log_int(rng, 1, 24), "hit": rng.choice([0.3, 0.6, 0.8, 0.95])}
    if kind == "beams":
        groups, fan = _log_int(rng, 1, 48), rng.choice([2, 3, 4, 8])
        n = _log_int(rng, 10, 4000)
        return {"op": "beams", "groups": groups, "fan": fan, "len_min": max(1, n // 3), "len_max": n, "page": page,
                "layers": rng.choice([1, 2, 3, 5]), "window": rng.choice([0, 0, 100, 1000]), "sinks": rng.choice([0, 4, 64])}
    return {"op": "copy", "pages": _log_int(rng, 1, 19200 // page), "page": page, "layers": _log_int(rng, 1, 8)}


def _spread(case, lo, hi, n, salt):
    """n sizes, log-uniform over lo..hi, from the case alone."""
    r = random.Random("%d %d %d %d %s" % (n, lo, hi, case["page"], salt))
    return [lo - 1 + _log_int(r, 1, hi - lo + 1) if lo < 64 else _log_int(r, lo, hi) for _ in range(n)]


def _lens(case):
    lens = _spread(case, case["len_min"], case["len_max"], case["batch"], "len")
    lens[0] = case["len_max"]
    return lens


def _trees(case):
    """(prefix lengths, nodes) of a finish case."""
    nodes = _spread(case, case["nodes_min"], case["nodes_max"], case["batch"], "nodes")
    return _spread(case, 1, max(1, case["len_max"] - 64), case["batch"], "past"), nodes


def _families(case):
    """(length of every branch, its parent) of a beams case: branches of a group have the same length."""
    lens = _spread(case, case["len_min"], case["len_max"], case["groups"], "beam")
    r = random.Random("%d %d %d parents" % (case["groups"], case["fan"], case["len_max"]))
    f = case["fan"]
    return [n for n in lens for _ in range(f)], [g * f + r.randrange(f) for g in range(case["groups"]) for _ in range(f)]


def _moves(case):
    """Rows that a finish case's walk moves, about: the walk goes on with probability hit from node to node, and a
    node's place is its own depth in few of the trees only."""
    h, a = case["hit"], case["accept"]
    return case["batch"] * min(a, sum(h ** i for i in range(1, a)))


def work(case):
    if case["op"] == "logprobs":
        n = case["rows"] * case["vocab"]
        size = 4 if case["type"] == "fp32" else 2
        return {"bytes": n * size + case["rows"] * (8 * case["given"] + 8 + 8 * case["top"]), "flops": 6 * n}
    if case["op"] == "window":
        lens = _lens(case)
        keys = sum(min(n, case["window"] + case["sinks"]) for n in lens)
        b, h = case["batch"], case["heads"]
        return {"bytes": keys * D_ROW * 2 + b * h * (D_ROW * 2 + D_LAT * 2 + 4) + -(-keys // case["page"]) * 4 + b * 4,
                "flops": 2 * h * keys * (D_ROW + D_LAT)}
    if case["op"] == "finish":
        past, nodes = _trees(case)
        return {"bytes": 12 * sum(nodes) + case["batch"] * (16 + 4 * case["accept"])
                + int(_moves(case)) * 2 * D_ROW * 2 * case["layers"], "flops": 0}
    if case["op"] == "beams":
        lens, parents = _families(case)
        page, layers = case["page"], case["layers"]
        cells = sum(-(-n // page) for n in lens)
        kept = len(set(parents))
        rows = sum(n % page for n in lens) * (1 - kept / len(parents))
        return {"bytes": cells * 8 + len(lens) * 24 + int(rows) * 2 * D_ROW * 2 * layers, "flops": 0}
    return {"bytes": case["pages"] * (case["page"] * D_ROW * 4 * case["layers"] + 12), "flops": 0}


# ------------------------------------------------------------------ inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _table(g, used, width, spare):
    """A table of the requests' pages in a random order, -1 behind them, and the number of pages."""
    total = sum(used)
    order = torch.randperm(total + spare, generator=g, device="cuda", dtype=torch.int32)
    have = torch.arange(width, device="cuda")[None, :] < torch.tensor(used, device="cuda")[:, None]
    table = torch.full((len(used), width), -1, dtype=torch.int32, device="cuda")
    table[have] = order[:total]
    return table, total + spare


def _prepare_logprobs(c, g):
    t, v = c["rows"], c["vocab"]
    store = torch.randn((t, v + c["pad"]), generator=g, device="cuda", dtype=TYPES[c["type"]]).mul_(2.5)
    x = store[:, :v]
    if c["masked"]:
        off = torch.rand((t, v), generator=g, device="cuda", dtype=torch.float32) < c["masked"]
        x.masked_fill_(off, -math.inf)
    tokens = torch.randint(0, v, (t, c["given"]), generator=g, device="cuda", dtype=torch.int32)
    f = lambda *n: torch.zeros(n, device="cuda")  # noqa: E731
    return {"logits": x, "tokens": tokens, "logprobs": f(t, c["given"]), "lse": f(t), "entropy": f(t),
            "top_ids": torch.zeros(t, c["top"], dtype=torch.int32, device="cuda"), "top_logprobs": f(t, c["top"])}


def _prepare_window(c, g):
    lens, page, b, h = _lens(c), c["page"], c["batch"], c["heads"]
    # pages that no position of the window or the sinks lies in were freed long ago: one number stands for them
    gone = [range(-(-c["sinks"] // page), max(0, n - c["window"]) // page) for n in lens]
    used = [-(-n // page) - len(x) for n, x in zip(lens, gone)]
    width = max(1, max(-(-n // page) for n in lens))
    packed, pages = _table(g, used, max(1, max(used)), 3)
    col = torch.arange(width, device="cuda")[None, :]
    first = torch.tensor([x.start for x in gone], device="cuda")[:, None]
    skip = torch.tensor([len(x) for x in gone], device="cuda")[:, None]
    at = torch.where(col < first, col, col - skip).clamp(0, packed.shape[1] - 1)
    table = torch.where((col >= first) & (col < first + skip), -1, packed.gather(1, at)).to(torch.int32).contiguous()
    cache = torch.randn((pages, page, D_ROW), generator=g, device="cuda", dtype=torch.bfloat16)
    return {"cache": cache, "table": table, "lens": _ints(lens),
            "q": torch.randn((b, h, D_ROW), generator=g, device="cuda", dtype=torch.bfloat16),
            "out": torch.zeros(b, h, D_LAT, dtype=torch.bfloat16, device="cuda"),
            "lse": torch.zeros(b, h, dtype=torch.float32, device="cuda")}


def _prepare_finish(c, g):
    past, nodes = _trees(c)
    page, b, most = c["page"], c["batch"], max(nodes)
    lens = [p + n for p, n in zip(past, nodes)]
    table, pages = _table(g, [-(-n // page) for n in lens], max(-(-n // page) for n in lens), 3)
    count = torch.tensor(nodes, device="cuda")
    i = torch.arange(most, device="cuda")
    real = i[None, :] < count[:, None]
    # node 0 hangs off the prefix, each other one off an earlier node near it, and the model chose every one's
    # token or, where it did not follow the draft, another
    back = 1 + (3 * torch.rand((b, most), generator=g, device="cuda") ** 2).long()
    parents = (i[None, :] - back).clamp_min(0)
    parents[:, 0] = -1
    tokens = torch.randint(0, 32000, (b, most), generator=g, device="cuda")
    targets = torch.randint(0, 32000, (b, most), generator=g, device="cuda")
    follows = torch.rand((b, most), generator=g, device="cuda") < c["hit"]
    follows[:, 0] = False
    tokens = torch.where(follows, targets.gather(1, parents.clamp_min(0)), tokens)
    first = tokens[:, 0].clone()
    # ancestors (the node itself among them), as the verify step had them for its mask
    ancestors = torch.eye(most, dtype=torch.bool, device="cuda").repeat(b, 1, 1)
    rows = torch.arange(b, device="cuda")
    for n in range(1, most):
        ancestors[:, n] |= ancestors[rows, parents[:, n]]
    z = lambda *n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    return {"cache": torch.randn((c["layers"], pages, page, D_ROW), generator=g, device="cuda", dtype=torch.bfloat16),
            "table": table, "lens": _ints(lens), "indptr": _ints([0] + nodes).cumsum(0).to(torch.int32),
            "parents": parents[real].to(torch.int32), "tokens": tokens[real].to(torch.int32),
            "targets": targets[real].to(torch.int32), "first": first.to(torch.int32), "ancestors": ancestors,
            "real": real, "path": z(b, c["accept"]), "counts": z(b), "next": z(b), "new_lens": z(b)}


def _prepare_beams(c, g):
    lens, parents = _families(c)
    page, f = c["page"], c["fan"]
    width = max(lens) // page + 2
    whole = [n // page for n in lens[::f]]  # pages that a group's branches share; the last is each one's own
    prefix, n0 = _table(g, whole, width, 0)
    table = prefix.repeat_interleave(f, 0)
    b = len(lens)
    held = [-(-n // page) for n in lens]
    tails = n0 + torch.randperm(b, generator=g, device="cuda", dtype=torch.int32)
    partial = torch.tensor([n % page > 0 for n in lens], device="cuda")
    rows = torch.arange(b, device="cuda")[partial]
    table[rows, torch.tensor(whole, device="cuda").repeat_interleave(f)[partial]] = tails[partial]
    pages = n0 + 3 * b + 5
    if c["window"]:  # what the window left behind in earlier steps is free; this one may leave a page more
        start = torch.tensor([max(0, n + 1 - c["window"] - page) // page for n in lens], device="cuda")[:, None]
        col = torch.arange(width, device="cuda")[None, :]
        table[(col >= -(-c["sinks"] // page)) & (col < start)] = -1
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    refs.index_add_(0, table[table >= 0].long(), torch.ones_like(table[table >= 0]))
    s = {"cache": torch.randn((c["layers"], pages, page, D_ROW), generator=g, device="cuda", dtype=torch.bfloat16),
         "tables": [table, torch.full_like(table, -1)], "held": [_ints(held), _ints(held)],
         "lens": [_ints(lens), _ints(lens)], "want": _ints([n + 1 for n in lens]), "parents": _ints(parents),
         "refs": refs, "copies": torch.zeros(b, 3, dtype=torch.int32, device="cuda"), "now": 0}
    return s


def _prepare_copy(c, g):
    n = c["pages"]
    order = torch.randperm(2 * n + 7, generator=g, device="cuda", dtype=torch.int32)
    cache = torch.randn((c["layers"], 2 * n + 7, c["page"], D_ROW), generator=g, device="cuda", dtype=torch.bfloat16)
    return {"cache": cache, "copies": torch.stack([order[:n], order[n:2 * n], torch.full_like(order[:n], c["page"])], 1)}


def prepare(case, seed):
    make = {"logprobs": _prepare_logprobs, "window": _prepare_window, "finish": _prepare_finish,
            "beams": _prepare_beams, "copy": _prepare_copy}[case["op"]]
    return {"case": dict(case), **make(case, _generator(seed))}


# ------------------------------------------------------- one pass, plainly

def _plain_logprobs(s):
    x = s["logits"].float()
    m = x.amax(-1, keepdim=True)
    d = x - m.clamp_min(-3e38)
    e = torch.exp(d)
    total = e.sum(-1)
    log_total = torch.log(total)
    lse = m.squeeze(-1) + log_total
    spread = torch.where(e > 0, e * d, 0.0).sum(-1) / total.clamp_min(1e-30)
    given = x.gather(1, s["tokens"].long()) - lse[:, None]
    # larger values first, then lower places: one whole number says both
    i = (x + 0.0).view(torch.int32)
    i = torch.where(i < 0, i ^ 0x7fffffff, i).long()
    key = (i << 32) - torch.arange(x.shape[1], device=x.device)
    ids = key.topk(s["case"]["top"], -1).indices
    return {"logprobs": given, "lse": lse, "entropy": log_total - spread, "top_ids": ids.to(torch.int32),
            "top_logprobs": x.gather(1, ids) - lse[:, None]}


def _plain_window(s):
    c, cache, lens = s["case"], s["cache"], s["lens"].long()
    page, n = c["page"], min(c["len_max"], c["window"] + c["sinks"])
    j = torch.arange(max(n, 1), device=cache.device)[None, :]
    start = (lens - c["window"]).clamp_min(0)[:, None]
    pos = torch.where((j < c["sinks"]) | (start <= c["sinks"]), j, start + j - c["sinks"])
    seen = pos < lens[:, None]
    pos = torch.where(seen, pos, 0)
    slot = s["table"].long().gather(1, pos // page) * page + pos % page
    rows = cache.view(-1, D_ROW)[slot.clamp_min(0)].float()
    sc = torch.matmul(s["q"].float(), rows.transpose(1, 2)) * SM_SCALE
    sc.masked_fill_(~seen[:, None, :], -math.inf)
    m = sc.amax(-1, keepdim=True).clamp_min(-1e30)
    p = torch.exp(sc.sub_(m))
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, rows[:, :, :D_LAT]) / total.clamp_min(1e-30)
    return {"out": out.to(cache.dtype), "lse": (m + torch.log(total)).squeeze(-1)}


def _plain_finish(s):
    c, cache, real, page = s["case"], s["cache"], s["real"], s["case"]["page"]
    b, most = real.shape
    i = torch.arange(most, device=cache.device)

    def padded(v):
        full = torch.full((b, most), -2, dtype=torch.int64, device=cache.device)
        full[real] = v.long()
        return full

    parents, tokens, targets = padded(s["parents"]), padded(s["tokens"]), padded(s["targets"])
    first = s["first"].long()
    want = torch.where(parents >= 0, targets.gather(1, parents.clamp_min(0)), first[:, None])
    hit = real & (tokens == want)
    earlier = (parents[:, :, None] == parents[:, None, :]) & hit[:, None, :] & (i[None, :] < i[:, None])
    hit = hit & ~earlier.any(-1)
    depth = s["ancestors"].sum(-1)
    taken = (s["ancestors"] & ~hit[:, None, :]).sum(-1) == 0
    taken = taken & real & (depth <= c["accept"])
    counts = taken.sum(-1)
    path = torch.full((b, c["accept"] + 1), -1, dtype=torch.int64, device=cache.device)
    path.scatter_(1, torch.where(taken, depth - 1, c["accept"]), torch.where(taken, i, -1))
    path = path[:, :-1]
    last = path.gather(1, (counts - 1).clamp_min(0)[:, None])
    nxt = torch.where(counts > 0, targets.gather(1, last.clamp_min(0)).squeeze(1), first)
    base = s["lens"].long() - real.sum(-1)
    move = path >= 0
    src, dst = base[:, None] + path, (base[:, None] + torch.arange(c["accept"], device=cache.device))
    req = torch.arange(b, device=cache.device)[:, None].expand_as(path)[move]
    src, dst = src[move], dst[move]
    table = s["table"].long()
    flat = cache.view(c["layers"], -1, D_ROW)
    flat[:, table[req, dst // page] * page + dst % page] = flat[:, table[req, src // page] * page + src % page]
    i32 = torch.int32
    return {"path": path.to(i32), "counts": counts.to(i32), "next": nxt.to(i32), "new_lens": (base + counts).to(i32),
            "cache": cache}


def _plain_beams(s):
    c, now, refs, cache, page = s["case"], s["now"], s["refs"], s["cache"], s["case"]["page"]
    old, held, lens = s["tables"][now], s["held"][now], s["lens"][now]
    new, parents = s["tables"][1 - now], s["parents"].long()
    b, width = old.shape
    col = torch.arange(width, device=cache.device)[None, :]
    one = torch.ones_like(parents, dtype=torch.int32)
    children = torch.zeros_like(one).index_add_(0, parents, one)
    there = (col < held[:, None]) & (old >= 0)
    refs.index_add_(0, old.clamp_min(0).long().view(-1), torch.where(there, children[:, None] - 1, 0).to(torch.int32).view(-1))
    held, lens = held[parents], lens[parents]
    table = torch.where(col < held[:, None], old[parents], new)
    # room for positions lens .. want - 1 in pages that nobody else holds
    ln, want = lens.long()[:, None], s["want"].long()[:, None]
    need = (want + page - 1) // page
    start = (ln + 1 - c["window"]).clamp_min(0) if c["window"] else torch.zeros_like(ln)
    there = (col < held[:, None]) & (table >= 0)
    cell = table.clamp_min(0).long()
    back = there & ((col >= need) | (col >= -(-c["sinks"] // page)) & (col < start // page))
    write = (col >= ln // page) & (col < need)
    shared = write & there & (refs[cell] > 1)
    left = refs.index_add(0, cell.view(-1), -(back | shared).to(torch.int32).view(-1))
    alone = shared & (left[cell] == 0)
    row = torch.arange(b, device=cache.device)[:, None].expand_as(cell)
    lowest = torch.full_like(refs, b, dtype=torch.int64).scatter_reduce_(
        0, cell.view(-1), torch.where(alone, row, b).view(-1), "amin")
    keep = alone & (lowest[cell] == row)
    left = left.index_add(0, cell.view(-1), keep.to(torch.int32).view(-1))
    take = write & (~there | shared & ~keep)
    free = (left == 0).cumsum(0)
    rank = take.view(-1).cumsum(0).view(b, width)
    enough = rank[-1, -1] <= free[-1]
    page_of = torch.searchsorted(free, rank).clamp_max(refs.shape[0] - 1)
    after = torch.where(take, page_of, torch.where(back, -1, table.long()))
    left = left.index_add(0, page_of.view(-1), take.to(torch.int32).view(-1))
    at = (ln // page).clamp_max(width - 1)
    copied = ((shared & ~keep).gather(1, at) & (ln % page > 0)).squeeze(1) & enough
    src, dst = table.gather(1, at).squeeze(1).long(), after.gather(1, at).squeeze(1)
    rows = (ln % page).squeeze(1)
    copies = torch.where(copied[:, None], torch.stack([src, dst, rows], 1), torch.tensor([-1, -1, 0], device=cache.device))
    new.copy_(torch.where(enough, after, table.long()))
    refs.copy_(torch.where(enough, left, refs))
    s["held"][1 - now].copy_(torch.where(enough, need.squeeze(1), held.long()))
    s["lens"][1 - now].copy_(lens)
    s["copies"].copy_(copies)
    s["now"] = 1 - now
    _plain_copy(s)
    return {"table": new, "held": s["held"][1 - now], "lens": s["lens"][1 - now], "refs": refs, "copies": s["copies"],
            "cache": cache}


def _plain_copy(s):
    cache, copies = s["cache"], s["copies"].long()
    which = copies[:, 1] >= 0
    src, dst, rows = copies[which].unbind(1)
    inside = torch.arange(cache.shape[2], device=cache.device)[None, :] < rows[:, None]
    cache[:, dst] = torch.where(inside[None, :, :, None], cache[:, src], cache[:, dst])
    return {"cache": cache}


# ---------------------------------------------------------- the same by calls

def _own_logprobs(abi, s):
    abi.mla_token_logprobs(s["logits"], s["tokens"], s["logprobs"], s["lse"], s["entropy"], s["top_ids"],
                           s["top_logprobs"])
    return {k: s[k] for k in ("logprobs", "lse", "entropy", "top_ids", "top_logprobs")}


def _own_window(abi, s):
    c = s["case"]
    if "workspace" not in s:
        s["workspace"] = torch.empty(abi.mla_paged_decode_workspace_bytes(c["batch"], c["heads"]), dtype=torch.uint8,
                                     device="cuda")
    abi.mla_paged_decode_window(s["q"], s["cache"], s["table"], s["lens"], c["window"], c["sinks"], SM_SCALE, s["out"],
                                s["lse"], s["workspace"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_finish(abi, s):
    abi.mla_tree_accept(s["parents"], s["tokens"], s["targets"], s["indptr"], s["lens"], s["path"], s["counts"],
                        s["next"], s["new_lens"], first=s["first"])
    abi.mla_paged_compact(s["path"], s["counts"], s["new_lens"], s["table"], s["cache"])
    return {k: s[k] for k in ("path", "counts", "next", "new_lens", "cache")}


def _own_beams(abi, s):
    c, a, b = s["case"], s["now"], 1 - s["now"]
    if "workspace" not in s:
        n = abi.mla_pages_fit_workspace_bytes(s["parents"].shape[0], s["refs"].shape[0])
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    abi.mla_pages_fork(s["parents"], s["lens"][a], s["held"][a], s["tables"][a], s["refs"], s["lens"][b], s["held"][b],
                       s["tables"][b])
    abi.mla_pages_fit(s["lens"][b], s["want"], s["held"][b], s["tables"][b], s["refs"], c["page"], s["copies"],
                      s["workspace"], window=c["window"], sinks=c["sinks"])
    abi.mla_paged_copy(s["copies"], s["cache"])
    s["now"] = b
    return {"table": s["tables"][b], "held": s["held"][b], "lens": s["lens"][b], "refs": s["refs"],
            "copies": s["copies"], "cache": s["cache"]}


def _own_copy(abi, s):
    abi.mla_paged_copy(s["copies"], s["cache"])
    return {"cache": s["cache"]}


def run(s):
    op = s["case"]["op"]
    if own:
        from speculative_decode_mla_tree_gb300 import abi
        return {"logprobs": _own_logprobs, "window": _own_window, "finish": _own_finish, "beams": _own_beams,
                "copy": _own_copy}[op](abi, s)
    return {"logprobs": _plain_logprobs, "window": _plain_window, "finish": _plain_finish, "beams": _plain_beams,
            "copy": _plain_copy}[op](s)


# ------------------------------------------------------- the same in 64 bits

def _exact_logprobs(c, s):
    parts = []
    for lo in range(0, c["rows"], 256):
        x = s["logits"][lo:lo + 256].double()
        lp = x - torch.logsumexp(x, -1, keepdim=True)
        ent = -torch.special.xlogy(lp.exp(), lp.exp()).sum(-1)
        values, ids = x.sort(dim=-1, descending=True, stable=True)
        k = c["top"]
        parts.append((lp.gather(1, s["tokens"][lo:lo + 256].long()), torch.logsumexp(x, -1), ent, ids[:, :k].int(),
                      lp.gather(1, ids[:, :k])))
    return dict(zip(("logprobs", "lse", "entropy", "top_ids", "top_logprobs"), (torch.cat(p) for p in zip(*parts))))


def _exact_window(c, s):
    flat, page = s["cache"].view(-1, D_ROW), c["page"]
    out = torch.zeros(c["batch"], c["heads"], D_LAT, dtype=torch.float64, device="cuda")
    lse = torch.full((c["batch"], c["heads"]), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(_lens(c)):
        near = torch.arange(max(0, n - c["window"]), n, device="cuda")
        far = torch.arange(0, min(c["sinks"], max(0, n - c["window"])), device="cuda")
        pos = torch.cat([far, near])
        if pos.numel() == 0:
            continue
        k = flat[s["table"][b].long()[pos // page] * page + pos % page].double()
        score = (s["q"][b].double() @ k.T) * SM_SCALE
        lse[b] = torch.logsumexp(score, -1)
        out[b] = torch.exp(score - lse[b][:, None]) @ k[:, :D_LAT]
    return {"out": out, "lse": lse}


def _exact_finish(c, s):
    past, nodes = _trees(c)
    par, tok, tar, first, table = (s[k].tolist() for k in ("parents", "tokens", "targets", "first", "table"))
    cache, page, at = s["cache"], c["page"], 0
    paths, counts, nxt, lens = [], [], [], []
    for b, n in enumerate(nodes):
        cur, want, path = -1, first[b], []
        while len(path) < c["accept"]:
            good = [i for i in range(n) if par[at + i] == cur and tok[at + i] == want]
            if not good:
                break
            cur = good[0]
            want = tar[at + cur]
            path.append(cur)
        for k, i in enumerate(path):  # in order: a row is read before another moves there
            p, q = past[b] + i, past[b] + k
            cache[:, table[b][q // page], q % page] = cache[:, table[b][p // page], p % page]
        paths.append(path + [-1] * (c["accept"] - len(path)))
        counts.append(len(path))
        nxt.append(want)
        lens.append(past[b] + len(path))
        at += n
    return {"path": _ints(paths), "counts": _ints(counts), "next": _ints(nxt), "new_lens": _ints(lens),
            "cache": cache.double()}


def _exact_beams(c, s):
    lens, parents = _families(c)
    page, old, b = c["page"], s["tables"][0].tolist(), len(lens)
    width = len(old[0])
    lens = [lens[p] for p in parents]
    rows = [list(old[p]) for p in parents]
    holders = {}
    for r, row in enumerate(rows):
        for p in row:
            if p >= 0:
                holders.setdefault(p, []).append(r)
    gone = -(-c["sinks"] // page)
    for r, row in enumerate(rows):
        start = max(0, lens[r] + 1 - c["window"]) if c["window"] else 0
        for j in range(gone, start // page):
            if row[j] >= 0:
                holders[row[j]].remove(r)
                row[j] = -1
    wanting = {}  # pages to be written, by those that want to
    for r, row in enumerate(rows):
        j = lens[r] // page
        if row[j] >= 0 and len(holders[row[j]]) > 1:
            wanting.setdefault(row[j], []).append(r)
    moving = {r: p for p, who in wanting.items() for r in who if len(who) < len(holders[p]) or r != min(who)}
    busy = {p for p, who in holders.items() if who}
    free = iter(p for p in range(s["refs"].shape[0]) if p not in busy)
    copies, cache = [], s["cache"]
    for r, row in enumerate(rows):
        j, n = lens[r] // page, lens[r] % page
        copies.append([-1, -1, 0])
        if r in moving:
            p = next(free)
            holders[row[j]].remove(r)
            holders[p] = [r]
            if n:
                copies[-1] = [row[j], p, n]
                cache[:, p, :n] = cache[:, row[j], :n]
            row[j] = p
        elif row[j] < 0:
            row[j] = next(free)
            holders[row[j]] = [r]
    refs = [len(holders.get(p, ())) for p in range(s["refs"].shape[0])]
    return {"table": _ints(rows), "held": _ints([n // page + 1 for n in lens]), "lens": _ints(lens), "refs": _ints(refs),
            "copies": _ints(copies), "cache": cache.double()}


def _exact_copy(c, s):
    cache = s["cache"].double()
    for src, dst, n in s["copies"].tolist():
        cache[:, dst, :n] = cache[:, src, :n]
    return {"cache": cache}


def exact(case, seed):
    s = prepare(case, seed)
    return {"logprobs": _exact_logprobs, "window": _exact_window, "finish": _exact_finish, "beams": _exact_beams,
            "copy": _exact_copy}[case["op"]](case, s)
