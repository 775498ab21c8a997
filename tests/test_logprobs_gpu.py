"""Log probabilities, entropy and most likely tokens on the GPU against their
definitions in 64 bits."""
import math

import pytest
import torch

import __graft_entry__
from speculative_decode_mla_tree_gb300 import abi

pytestmark = pytest.mark.gpu
F32_HALF = 2.0 ** -24
INF, NAN = math.inf, math.nan
TYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    __graft_entry__.build()


def call(x, tokens, k, entropy=True, status=None):
    t = x.shape[0]
    z = lambda *n: torch.full(n, 77.0, device="cuda")  # noqa: E731
    lp = None if tokens is None else z(*tokens.shape)
    out = {"lse": z(t), "entropy": z(t) if entropy else None, "lp": lp,
           "ids": torch.full((t, k), -77, dtype=torch.int32, device="cuda"), "top": z(t, k)}
    abi.mla_token_logprobs(x, None if tokens is None else tokens.cuda(), lp, out["lse"], out["entropy"],
                           out["ids"] if k else None, out["top"] if k else None, status)
    return {n: v.cpu() for n, v in out.items() if v is not None}


def reference(x, tokens, k):
    """In 64 bits, and how far fp32 may be off: see the bounds."""
    x = x.double()
    m = x.amax(-1, keepdim=True)
    none = torch.isneginf(m.squeeze(-1))
    odd = ~torch.isfinite(m.squeeze(-1)) & ~none
    log_s = torch.logsumexp(x - m, -1)  # apart from m, beside which it may vanish in 64 bits, too
    lse = m.squeeze(-1) + log_s
    lse[odd] = NAN
    p = torch.exp(x - m - log_s[:, None])
    d = torch.where(p > 0, x - m, torch.zeros_like(x))
    ent = log_s - (p * d).sum(-1)
    ent[odd] = NAN
    ent[none] = 0.0
    ids = torch.where(torch.isnan(x), NAN, x).sort(dim=-1, descending=True, stable=True).indices[:, :k]  # one kind of NaN
    lse[none] = -INF

    def lp_of(v):
        r = v - lse[:, None]
        r[none] = -INF
        return r

    # Relative error of a sum of exp: every term's own (exp2 to two units, its argument's
    # two roundings, so 2^-23 of the exponent, on average over the terms), and an
    # addition's for at most vocab / 128 values of a thread one after another and the joins.
    y = (p * d.abs()).sum(-1).nan_to_num(0.0) / math.log(2) + 1  # (rows without a finite sum are compared exactly)
    rel = (8 + 4 * y + x.shape[1] / 128 + 64) * F32_HALF
    # ln, the maximum's addition and one rounding
    lse_tol = rel + 4 * F32_HALF * (lse.abs() + 1)
    # ln S and T / S, T a sum of the same terms times the exponent: of the same relative error twice
    ent_tol = rel * (2 + 3 * y) + 4 * F32_HALF * (ent.abs() + 1)
    want = {"lse": lse, "entropy": ent, "ids": ids.int(), "top": lp_of(x.gather(1, ids))}
    tol = {"lse": lse_tol, "entropy": ent_tol}
    tol["top"] = lse_tol[:, None] + 2 * F32_HALF * want["top"].abs().nan_to_num(0, 0, 0)
    if tokens is not None:
        t = tokens.long().view(x.shape[0], -1).cuda()
        lp = lp_of(x.gather(1, t.clamp(0, x.shape[1] - 1)))
        lp[(t < 0) | (t >= x.shape[1])] = -INF
        want["lp"] = lp.view(tokens.shape)
        tol["lp"] = (lse_tol[:, None] + 2 * F32_HALF * lp.abs().nan_to_num(0, 0, 0)).view(tokens.shape)
    return {n: v.cpu() for n, v in want.items()}, {n: v.cpu() for n, v in tol.items()}


def check(x, tokens, k, status=None):
    got = call(x, tokens, k, status=status)
    want, tol = reference(x, tokens, k)
    assert torch.equal(got["ids"], want["ids"])
    for n, t in tol.items():
        g, w = got[n].double(), want[n].clone()
        w[w < -torch.finfo(torch.float32).max] = -INF  # no fp32 number is as low
        assert torch.equal(torch.isnan(g), torch.isnan(w)), n
        fine = torch.isfinite(w)
        assert torch.equal(torch.isfinite(g), fine), n
        assert torch.equal(g[~fine & ~torch.isnan(w)], w[~fine & ~torch.isnan(w)]), n
        off = (g - w).abs()
        t = torch.broadcast_to(t, g.shape)
        assert (off[fine] <= t[fine]).all(), (n, float((off[fine] / t[fine]).max()))
    return got


def rows(seed, t, v, dtype, scale=3.0, pad=0, shift=0):
    """[t, v] of a row stride v + pad whose first element is `shift` elements into its memory."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    store = torch.full((t * (v + pad) + shift,), NAN, dtype=dtype, device="cuda")
    x = store[shift:].view(t, v + pad)[:, :v]
    x.copy_(torch.randn(t, v, generator=g, device="cuda") * scale)
    return x, torch.randint(0, v, (t,), generator=g, dtype=torch.int32, device="cuda").cpu()


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("v", [1, 2, 3, 7, 8, 9, 31, 33, 100, 255, 256, 257, 511, 513, 2047, 2049, 8191, 20011, 65536])
def test_sizes(dtype, v):
    x, tok = rows(v, 5, v, dtype, pad=v % 3, shift=v % 5)
    for k in sorted({1, 2, 5, 8, 20, 32}):
        if k <= v:
            check(x, tok, k)
    check(x, tok[:, None].repeat(1, 3), 0)


@pytest.mark.parametrize("t,v,dtype", [(1, 151000, torch.bfloat16), (3, 262147, torch.float32), (40, 50001, torch.float16),
                                       (200, 40000, torch.bfloat16), (700, 40000, torch.bfloat16), (1300, 3001, torch.float32),
                                       (1300, 20001, torch.float32), (2500, 33, torch.bfloat16)])
@pytest.mark.parametrize("k", [1, 8, 9, 32])
def test_rows(t, v, dtype, k):
    """Every split of a row, and every block size."""
    x, tok = rows(t + k, t, v, dtype, pad=1)
    check(x, tok, k)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("v", [1, 5, 8, 31, 127, 255, 256, 257, 264, 1000, 2047, 4001, 8192])
def test_many_short_rows(dtype, v):
    """More rows than blocks that run at once, of one warp each for the shortest."""
    x, tok = rows(v, 1300, v, dtype, pad=v % 3, shift=v % 5)
    for k in (0, 1, 8, 9, 20, 21, 32):
        if k <= v:
            check(x, tok, k)


@pytest.mark.parametrize("t", [300, 310, 450, 470, 600, 610])
@pytest.mark.parametrize("v,dtype", [(999, torch.bfloat16), (32768, torch.bfloat16), (33001, torch.float16), (20001, torch.float32)])
def test_two_to_four_blocks_a_multiprocessor(t, v, dtype):
    x, tok = rows(t, t, v, dtype, pad=3)
    for k in (0, 5, 20, 21):
        check(x, tok, k)


SPECIAL = {
    "all masked": lambda x: x.fill_(-INF),
    "one left": lambda x: x[:, 1:].fill_(-INF),
    "last left": lambda x: x[:, :-1].fill_(-INF),
    "few left": lambda x: x[:, 3:-2].fill_(-INF),
    "every 17th": lambda x: x.masked_fill_(torch.arange(x.shape[1], device="cuda") % 17 != 3, -INF),
    "lowest masks": lambda x: x[:, 5:].fill_(torch.finfo(x.dtype).min),
    "all lowest": lambda x: x.fill_(torch.finfo(x.dtype).min),
    "lowest and masked": lambda x: (x.fill_(torch.finfo(x.dtype).min), x[:, ::3].fill_(-INF)),
    "all largest": lambda x: x.fill_(torch.finfo(x.dtype).max),
    "largest and lowest": lambda x: (x.fill_(torch.finfo(x.dtype).max), x[:, ::3].fill_(torch.finfo(x.dtype).min)),
    "all equal": lambda x: x.fill_(1.5),
    "zeros of both signs": lambda x: (x.fill_(0.0), x[:, ::2].fill_(-0.0)),
    "two values": lambda x: x.copy_((x > 0).to(x.dtype)),
    "rising": lambda x: x.copy_(torch.arange(x.shape[1], device="cuda") / 64.0),
    "falling": lambda x: x.copy_(-torch.arange(x.shape[1], device="cuda") / 64.0),
    "large in one thread": lambda x: x.add_(torch.where(torch.arange(x.shape[1], device="cuda") // 8 % 64 == 5, 20.0, 0.0)),
    "large in half the warps": lambda x: x.add_(torch.where(torch.arange(x.shape[1], device="cuda") // 256 % 2 == 1, 30.0, 0.0)),
    "far apart": lambda x: x.mul_(1000.0),
    "high": lambda x: x.add_(30000.0),
}


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("v", [13, 300, 40000])
@pytest.mark.parametrize("name", SPECIAL)
def test_special_rows(name, v, dtype):
    for t in (2, 700):
        x, tok = rows(1, t, v, dtype, shift=3)
        SPECIAL[name](x)
        for k in (1, 7, 13):
            check(x, tok, k)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("v", [13, 300, 2000])
@pytest.mark.parametrize("name", SPECIAL)
def test_special_rows_among_many(name, v, dtype):
    """Every third row, so that others of the same launch see that nothing spills over."""
    x, tok = rows(6, 1500, v, dtype, shift=1)
    y = x[::3].clone()
    SPECIAL[name](y)
    x[::3] = y
    x[4] = NAN
    x[5, v // 2], x[7, 1] = INF, NAN
    for k in (1, 8, 13):
        check(x, tok, k)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("v", [13, 40000])
@pytest.mark.parametrize("what", [NAN, -NAN, INF])
def test_nan_and_inf(v, dtype, what):
    """Rows that hold them say so, in all but the order of their tokens; the others do not notice."""
    x, tok = rows(2, 9, v, dtype, pad=3)
    x[1, 0] = what
    x[3, v - 1] = what
    x[5, v // 2] = what
    x[5, v // 3] = -INF
    x[7] = what
    for k in (1, 13):
        got = check(x, tok, k)
    assert torch.isnan(got["lse"][[1, 3, 5, 7]]).all() and torch.isfinite(got["lse"][[0, 2, 4, 6, 8]]).all()


def test_tokens_out_of_range():
    x, _ = rows(3, 4, 1000, torch.bfloat16)
    tok = torch.tensor([[0, -1, 999], [-1, -1, -1], [5, 6, 7], [1, 1, 1]], dtype=torch.int32)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    check(x, tok, 3, status)
    assert int(status) == 0
    tok[2, 0], tok[3, 2] = 1000, -2
    check(x, tok, 3, status)
    assert int(status) == abi.DEV_BAD_TOKEN
    many = torch.randint(-1, 1000, (4, 300), dtype=torch.int32)
    check(x, many, 3)


def test_layouts():
    """Rows apart, overlapping and the same, a column of tokens, outputs left out."""
    x, tok = rows(4, 6, 5000, torch.bfloat16, pad=13, shift=1)
    wide = torch.zeros(6, 4, dtype=torch.int32)
    wide[:, 2] = tok
    lp = torch.zeros(6, device="cuda")
    abi.mla_token_logprobs(x, wide.cuda()[:, 2], lp)
    want, tol = reference(x, tok, 1)
    assert ((lp.cpu().double() - want["lp"]).abs() <= tol["lp"]).all()
    same = x[:1].expand(6, 5000)
    check(same, tok, 4)
    sliding = x.as_strided((6, 5000), (1, 1))
    sliding.nan_to_num_(0.0)
    check(sliding, tok, 4)
    ids = torch.zeros(6, 2, dtype=torch.int32, device="cuda")
    abi.mla_token_logprobs(x, top_ids=ids)
    assert torch.equal(ids.cpu(), reference(x, None, 2)[0]["ids"])
    abi.mla_token_logprobs(x[:0], tok[:0].cuda(), lp[:0])
    abi.mla_token_logprobs(x)


def test_same_in_every_run_and_in_a_graph():
    x, tok = rows(5, 30, 50000, torch.bfloat16)
    first = call(x, tok, 20)
    t = x.shape[0]
    s = torch.cuda.Stream()
    lp, lse, ent = torch.zeros(t, device="cuda"), torch.zeros(t, device="cuda"), torch.zeros(t, device="cuda")
    ids, top = torch.zeros(t, 20, dtype=torch.int32, device="cuda"), torch.zeros(t, 20, device="cuda")
    tc, xc = tok.cuda(), torch.zeros_like(x)
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            abi.mla_token_logprobs(xc, tc, lp, lse, ent, ids, top)
    torch.cuda.synchronize()
    xc.copy_(x)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(lp.cpu(), first["lp"]) and torch.equal(lse.cpu(), first["lse"])
        assert torch.equal(ent.cpu(), first["entropy"]) and torch.equal(ids.cpu(), first["ids"])
        assert torch.equal(top.cpu(), first["top"])


def test_binding_refuses():
    x, tok = rows(6, 4, 100, torch.bfloat16)
    tok, lp = tok.cuda(), torch.zeros(4, device="cuda")
    ids = torch.zeros(4, 3, dtype=torch.int32, device="cuda")
    bad = [
        (dict(logits=x.cpu()), "logits must be a CUDA tensor"), (dict(logits=x.double()), "bf16, fp16 or fp32"),
        (dict(logits=x[0]), "logits must be .* 2 dimensions"), (dict(logits=x[:, ::2]), "unit stride"),
        (dict(logits=x[:, :0]), "vocabulary"), (dict(tokens=tok.long()), "tokens must be torch.int32"),
        (dict(tokens=tok[:3]), "rows"), (dict(logprobs=None), "go together"), (dict(tokens=None), "go together"),
        (dict(logprobs=lp.double()), "logprobs must be"), (dict(logprobs=lp[:3]), "logprobs must be"),
        (dict(lse=lp[:2]), "lse must be"), (dict(entropy=torch.zeros(8, device="cuda")[::2]), "contiguous"),
        (dict(top_ids=ids.long()), "top_ids must be"), (dict(top_ids=ids.t()), "top_ids"),
        (dict(top_logprobs=torch.zeros(4, 3, device="cuda")), "needs top_ids"),
        (dict(top_ids=ids, top_logprobs=torch.zeros(4, 2, device="cuda")), "top_logprobs must be"),
        (dict(status=lp), "status must be"), (dict(top_ids=torch.zeros(4, 33, dtype=torch.int32, device="cuda")), "unsupported"),
    ]
    for kw, message in bad:
        with pytest.raises(abi.MlaTreeError, match=message):
            abi.mla_token_logprobs(**{**dict(logits=x, tokens=tok, logprobs=lp), **kw})
    with pytest.raises(abi.MlaTreeError, match="invalid"):
        abi.mla_token_logprobs(x[:, :2], top_ids=ids)
