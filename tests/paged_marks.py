"""Keys that can be told apart in a decode result.

With all scores equal, an output is the plain mean of the values. Every key has
the value 1 in one of the 512 dims and 0 in the others, the dims dealt out in a
shuffled order, so that out[d] * n is the number of keys with dim d: whole, and
below 128 for up to 50000 keys, where half a step of bf16 (2^-8 of the value at
most) still tells the numbers apart. A key that is lost, counted twice or taken
for another one changes a number; lse = ln n shows how many there are."""
import math

import torch

import paged_ref as ref

MAX_KEYS = 50000


def marked(g, n):
    """(values [n, 512], keys per dim [512]): dims dealt out evenly, shuffled."""
    assert n <= MAX_KEYS  # at most 98 keys a dim
    dim = (torch.randperm(n, generator=g) % 512)
    v = torch.zeros(n, 512)
    v[torch.arange(n), dim] = 1.0
    return v, torch.bincount(dim, minlength=512)


def check_marks(out, lse, n, counts):
    """out [heads, 512], lse [heads] of a request with n marked keys, all scores 0.
    out is off by half a step of bf16 and, in fp32, by one truncated sum of a
    16-key step after another (n / 16 + 64 of 2^-23): together less than half a
    key. lse is ln of a sum of n ones, exact in fp32, to a few units in the last
    place (16 half steps: a key more or less is 1 / n, twice that at 50000)."""
    assert 98 * (ref.BF16_HALF + (n / 16 + 64) * 2 * ref.F32_HALF) < 0.5
    got = out.double() * n
    assert torch.equal(got.round().long(), counts.expand_as(got)), (got - counts).abs().max()
    assert ((got - counts).abs() < 0.45).all()
    assert ((lse.double() - math.log(n)).abs() <= 16 * ref.F32_HALF * (1 + math.log(n))).all()


def check_close(out, lse, want_out, want_lse):
    """Results of 1000 keys and more against 64 bits by their usual error, for
    normal keys and queries of half that size (scores of 0.87 in nats, so half
    the keys count). Rows of 512 outputs in the 2-norm: a value rounded to bf16
    is off by 1.66e-3 of itself (root mean square over evenly spread logarithms:
    half a step over sqrt(3), times 0.7355), the weights by as much each, which
    moves an average of independent values alike: sqrt(2) x 1.66e-3 = 2.35e-3,
    a quarter more allowed. lse: a score's 36 fp32 sums of 16 products, each
    truncated at 2^-23 of three deviations of the unscaled score (36) at most,
    times the scale of 0.072: 1.1e-5, beside half steps of lse itself."""
    err = (out.double() - want_out).norm(dim=-1) / want_out.norm(dim=-1)
    assert (err <= 2.95e-3).all(), err.max()
    off = (lse.double() - want_lse).abs()
    assert (off <= 1.1e-5 + 8 * ref.F32_HALF * want_lse.abs()).all(), off.max()
