"""Cases of the paged-cache operators of a latent-attention serving step.

* append: new tokens' key-value rows go into a paged latent cache, the latent
  part normalised where the model does so, the rope part rotated to the token's
  position, and the queries' rope part rotated next to it.
* decode: attention of one new token per request over that cache, split over
  the cache's length and joined.

``run`` computes them in plain torch operations, or, where ``own`` is set, by
the library's entry points. A cache row is 576 bf16 values (512 latent, 64
rope); a page holds ``page`` rows; ``block_table[b, j]`` is the page of request
b's positions ``j * page ..``; ``kv_lens[b]`` is its length with the new tokens.
"""
import math
import random

import torch

own = False

D_LAT, D_ROPE, D_ROW = 512, 64, 576
SM_SCALE = 1.0 / math.sqrt(192.0)
EPS = 1e-6


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one sequence generating a token, a head-parallel shard of 8 heads: latency alone counts
        {"name": "append_one_token", "op": "append", "batch": 1, "new_min": 1, "new_max": 1, "past_min": 21,
         "past_max": 21, "heads": 8, "page": 64, "style": "pairs", "norm": True, "depths": False},
        # the draft tree of a verify step: rope positions are tree depths, rows go one after another; small pages
        {"name": "append_draft_trees", "op": "append", "batch": 8, "new_min": 16, "new_max": 16, "past_min": 1024,
         "past_max": 4096, "heads": 8, "page": 16, "style": "halves", "norm": False, "depths": True},
        # a large generation batch, one token each
        {"name": "append_generation_batch", "op": "append", "batch": 256, "new_min": 1, "new_max": 1, "past_min": 0,
         "past_max": 2047, "heads": 64, "page": 32, "style": "pairs", "norm": True, "depths": False},
        # prompts of odd lengths, taken in one ragged batch
        {"name": "append_prompts", "op": "append", "batch": 7, "new_min": 333, "new_max": 2111, "past_min": 0,
         "past_max": 1000, "heads": 64, "page": 64, "style": "pairs", "norm": True, "depths": False},
        # the logged single request: 30 keys, 8 heads
        {"name": "decode_short", "op": "decode", "batch": 1, "len_min": 30, "len_max": 30, "heads": 8, "page": 64},
        # a few chats on a shard of 8 heads
        {"name": "decode_small_batch", "op": "decode", "batch": 8, "len_min": 1024, "len_max": 4096, "heads": 8,
         "page": 64},
        # a ragged odd batch with empty slots in it, small pages, a head count that fills no tile
        {"name": "decode_ragged_odd", "op": "decode", "batch": 37, "len_min": 0, "len_max": 5001, "heads": 24,
         "page": 16},
        # 64 heads at 8192 keys
        {"name": "decode_batch", "op": "decode", "batch": 32, "len_min": 8192, "len_max": 8192, "heads": 64, "page": 64},
        # all 128 heads of a large model on one card (data-parallel attention)
        {"name": "decode_all_heads", "op": "decode", "batch": 48, "len_min": 2000, "len_max": 16384, "heads": 128,
         "page": 32},
        # one document of 131071 tokens: everything rests on the split over the length
        {"name": "decode_one_long", "op": "decode", "batch": 1, "len_min": 131071, "len_max": 131071, "heads": 64,
         "page": 128},
        # four sequences of 200000 keys, 16 heads
        {"name": "decode_long", "op": "decode", "batch": 4, "len_min": 200000, "len_max": 200000, "heads": 16,
         "page": 64},
        # the 64-request serving mix: lengths 128 to 131072, log-uniform
        {"name": "decode_mix", "op": "decode", "batch": 64, "len_min": 128, "len_max": 131072, "heads": 64, "page": 64},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    heads = rng.choice([_log_int(rng, 1, 128), rng.choice([8, 16, 32, 64, 128])])
    page = rng.choice([8, 16, 32, 64, 128, 256])
    if rng.random() < 0.4:
        batch = _log_int(rng, 1, 256)
        new_max = _log_int(rng, 1, max(1, 7000 // batch))
        past = _log_int(rng, 1, max(1, 300000 // batch if batch > 8 else 32768))
        return {"op": "append", "batch": batch, "new_min": max(1, new_max // rng.choice([1, 2, 5])), "new_max": new_max,
                "past_min": 0, "past_max": past, "heads": min(heads, 64), "page": page,
                "style": rng.choice(["pairs", "halves"]), "norm": rng.random() < 0.5, "depths": rng.random() < 0.3}
    batch = _log_int(rng, 1, 128)
    len_max = _log_int(rng, 1, 600000 // max(batch, 5))
    return {"op": "decode", "batch": batch, "len_min": rng.choice([0, len_max // 7, len_max]), "len_max": len_max,
            "heads": heads, "page": page}


def _spread(case, lo, hi, salt):
    """One length per request, log-uniform over lo..hi, from the case alone."""
    r = random.Random("%d %d %d %d %s" % (case["batch"], lo, hi, case["heads"], salt))
    out = [lo - 1 + _log_int(r, 1, hi - lo + 1) if lo < 64 else _log_int(r, lo, hi) for _ in range(case["batch"])]
    return out


def _sizes(case):
    """(new tokens, lengths with them) of every request."""
    if case["op"] == "decode":
        lens = _spread(case, case["len_min"], case["len_max"], "len")
        lens[0] = case["len_max"]
        return [1] * len(lens), lens
    new = _spread(case, case["new_min"], case["new_max"], "new")
    past = _spread(case, case["past_min"], case["past_max"], "past")
    return new, [n + p for n, p in zip(new, past)]


def work(case):
    new, lens = _sizes(case)
    t, h, b = sum(new), case["heads"], case["batch"]
    if case["op"] == "append":
        # rows and rope queries in and out, the angles' cosines and sines, and one page number per page written
        pages = sum(-(-n // case["page"]) for n in new)
        return {"bytes": t * (2 * D_ROW * 2 + 2 * h * D_ROPE * 2 + D_ROPE * 4) + pages * 4 + b * 8
                + (D_LAT * 2 if case["norm"] else 0), "flops": t * (3 * D_ROPE * (h + 1) + (4 * D_LAT if case["norm"] else 0))}
    keys, pages = sum(lens), sum(-(-n // case["page"]) for n in lens)
    return {"bytes": keys * D_ROW * 2 + b * h * (D_ROW * 2 + D_LAT * 2 + 4) + pages * 4 + b * 4,
            "flops": 2 * h * keys * (D_ROW + D_LAT)}


# ------------------------------------------------------------------ inputs

def _rope_table(n, dev):
    """cos | sin of position * 10000^(-i / 32), i < 32, as a serving program keeps them."""
    f = torch.exp(torch.arange(D_ROPE // 2, dtype=torch.float64, device=dev) * (-math.log(10000.0) * 2 / D_ROPE))
    a = torch.arange(n, dtype=torch.float64, device=dev)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.bfloat16)

    new, lens = _sizes(case)
    b, h, page, t = case["batch"], case["heads"], case["page"], sum(new)
    width = max(1, -(-max(lens) // page))
    used = [-(-n // page) for n in lens]
    pages = sum(used) + 3
    order = torch.randperm(pages, generator=g, device=dev, dtype=torch.int32)
    have = torch.arange(width, device=dev)[None, :] < torch.tensor(used, device=dev)[:, None]
    table = torch.zeros(b, width, dtype=torch.int32, device=dev)
    table[have] = order[:sum(used)]
    s = {"case": dict(case), "cache": normal(pages, page, D_ROW), "table": table,
         "lens": torch.tensor(lens, dtype=torch.int32, device=dev)}
    if case["op"] == "decode":
        s["q"] = normal(b, h, D_ROW)
        s["out"] = torch.zeros(b, h, D_LAT, dtype=torch.bfloat16, device=dev)
        s["lse"] = torch.zeros(b, h, dtype=torch.float32, device=dev)
        return s
    # one projection's output holds the latent and the rope key side by side, another the queries (128 + 64 a head)
    s["row"] = normal(t, D_ROW)
    s["proj_q"] = normal(t, h, 192)
    s["q"] = normal(t, h, D_ROW)
    s["indptr"] = torch.tensor([0] + new, device=dev).cumsum(0).to(torch.int32)
    s["rope"] = _rope_table(max(lens), dev)
    s["weight"] = (1 + 0.1 * normal(D_LAT).float()).to(torch.bfloat16) if case["norm"] else None
    s["pos"] = None
    if case["depths"]:  # a chain of drafts with siblings: depths at most the row's own place
        own_place = torch.cat([torch.arange(n, device=dev) for n in new])
        past = torch.tensor([le - n for n, le in zip(new, lens)], device=dev).repeat_interleave(torch.tensor(new, device=dev))
        s["pos"] = (past + (own_place * torch.rand(t, generator=g, device=dev)).long()).to(torch.int32)
    return s


# ------------------------------------------------------------------ one pass

def _rotate(x, cos, sin, style):
    """x [..., 64] in 32 bits, cos and sin [..., 32] of its pairs."""
    if style == "pairs":
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    a, b = x[..., :32], x[..., 32:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _plain_append(s):
    c, indptr, lens, cache, page = s["case"], s["indptr"].long(), s["lens"].long(), s["cache"], s["case"]["page"]
    t = s["row"].shape[0]
    tok = torch.arange(t, device=cache.device)
    req = torch.searchsorted(indptr, tok, right=True) - 1
    place = lens[req] - indptr[req + 1] + tok
    pos = place if s["pos"] is None else s["pos"].long()
    cos, sin = s["rope"][pos, :32], s["rope"][pos, 32:]
    lat = s["row"][:, :D_LAT].float()
    if s["weight"] is not None:
        lat = lat * torch.rsqrt((lat * lat).mean(-1, keepdim=True) + EPS) * s["weight"].float()
    key = _rotate(s["row"][:, D_LAT:].float(), cos, sin, c["style"])
    slot = s["table"][req, place // page].long() * page + place % page
    cache.view(-1, D_ROW)[slot] = torch.cat([lat, key], 1).to(cache.dtype)
    s["q"][:, :, D_LAT:] = _rotate(s["proj_q"][:, :, 128:].float(), cos[:, None], sin[:, None], c["style"]).to(cache.dtype)
    return {"cache": cache, "q": s["q"]}


def _plain_decode(s):
    cache, lens, page = s["cache"], s["lens"].long(), s["case"]["page"]
    n = int(s["case"]["len_max"])
    j = torch.arange(max(n, 1), device=cache.device)
    slot = s["table"].long()[:, j // page] * page + j % page
    rows = cache.view(-1, D_ROW)[slot].float()
    seen = j[None, :] < lens[:, None]
    sc = torch.matmul(s["q"].float(), rows.transpose(1, 2)) * SM_SCALE
    sc.masked_fill_(~seen[:, None, :], -math.inf)
    m = sc.amax(-1, keepdim=True).clamp_min(-1e30)
    p = torch.exp(sc.sub_(m))
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, rows[:, :, :D_LAT]) / total.clamp_min(1e-30)
    lse = (m + torch.log(total)).squeeze(-1)
    return {"out": out.to(cache.dtype), "lse": lse}


def run(s):
    c = s["case"]
    if own:
        from speculative_decode_mla_tree_gb300 import abi
        if c["op"] == "append":
            abi.mla_paged_append(s["row"][:, :D_LAT], s["row"][:, D_LAT:], s["indptr"], s["lens"], s["table"], s["cache"],
                                 s["rope"], q_rope=s["proj_q"][:, :, 128:], q_out=s["q"][:, :, D_LAT:], positions=s["pos"],
                                 norm_weight=s["weight"], norm_eps=EPS,
                                 rope_style=abi.ROPE_PAIRS if c["style"] == "pairs" else abi.ROPE_HALVES)
            return {"cache": s["cache"], "q": s["q"]}
        if "workspace" not in s:
            n = abi.mla_paged_decode_workspace_bytes(c["batch"], c["heads"])
            s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
        abi.mla_paged_decode(s["q"], s["cache"], s["table"], s["lens"], SM_SCALE, s["out"], s["lse"], s["workspace"])
        return {"out": s["out"], "lse": s["lse"]}
    return _plain_append(s) if c["op"] == "append" else _plain_decode(s)


# ------------------------------------------------------- the same in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    new, lens = _sizes(case)
    page, table = case["page"], s["table"].tolist()
    flat = s["cache"].double().reshape(-1, D_ROW) if case["op"] == "append" else s["cache"].reshape(-1, D_ROW)

    def slots(b, lo, hi):
        first, last = lo // page, -(-hi // page)
        ids = torch.tensor(table[b][first:last], dtype=torch.int64, device=flat.device)
        every = (ids[:, None] * page + torch.arange(page, device=flat.device)).reshape(-1)
        return every[lo - first * page:hi - first * page]

    if case["op"] == "decode":
        out = torch.zeros(case["batch"], case["heads"], D_LAT, dtype=torch.float64, device=flat.device)
        lse = torch.full((case["batch"], case["heads"]), -math.inf, dtype=torch.float64, device=flat.device)
        for b, n in enumerate(lens):
            if n == 0:
                continue
            k = flat[slots(b, 0, n)].double()
            score = (s["q"][b].double() @ k.T) * SM_SCALE
            lse[b] = torch.logsumexp(score, -1)
            out[b] = torch.exp(score - lse[b][:, None]) @ k[:, :D_LAT]
        return {"out": out, "lse": lse}

    q = s["q"].double()
    at = 0
    i = torch.arange(D_ROPE // 2, device=flat.device)
    one, two = (2 * i, 2 * i + 1) if case["style"] == "pairs" else (i, i + D_ROPE // 2)
    for b, (n, le) in enumerate(zip(new, lens)):
        if n == 0:
            continue
        rows = s["row"][at:at + n].double()
        pos = torch.arange(le - n, le, device=flat.device) if s["pos"] is None else s["pos"][at:at + n].long()
        ang = s["rope"][pos].double()  # the table is an input: its values are taken as they are
        turn = torch.complex(ang[:, :32], ang[:, 32:])
        if s["weight"] is not None:
            lat = rows[:, :D_LAT]
            rows[:, :D_LAT] = lat / (lat.square().sum(-1, keepdim=True) / D_LAT + EPS).sqrt() * s["weight"].double()
        z = torch.complex(rows[:, D_LAT + one], rows[:, D_LAT + two]) * turn
        rows[:, D_LAT + one], rows[:, D_LAT + two] = z.real, z.imag
        flat[slots(b, le - n, le)] = rows
        pq = s["proj_q"][at:at + n].double()
        z = torch.complex(pq[:, :, 128 + one], pq[:, :, 128 + two]) * turn[:, None]
        q[at:at + n, :, D_LAT + one], q[at:at + n, :, D_LAT + two] = z.real, z.imag
        at += n
    return {"cache": flat.reshape(s["cache"].shape), "q": q}
