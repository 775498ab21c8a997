"""The checks of paged_marks accept what a right kernel gives and refuse results
with keys lost, doubled or exchanged (mistakes planted in the 64-bit oracle)."""
import math

import pytest
import torch

import paged_marks as marks

N = [1000, 12000, 20011]


def attend(q, keys, weight, scale):
    """out [heads, 512] in bf16, lse [heads] in fp32; weight: how often each key counts."""
    s = q.double() @ keys.double().T * scale + torch.log(weight.double())
    lse = torch.logsumexp(s, -1)
    return (torch.exp(s - lse[:, None]) @ keys[:, :512].double()).bfloat16(), lse.float()


def mistakes(n):
    def lost(*rows):
        w = torch.ones(n)
        for r in rows:
            w[r] = 0
        return w

    def doubled(r):
        w = torch.ones(n)
        w[r] = 2
        return w

    tile = 64 * (n // 128)
    both = lost(slice(tile, tile + 64))
    both[tile - 64:tile] = 2
    last = 64 * ((n - 1) // 64)
    return {"first key": lost(0), "last key": lost(n - 1), "last three": lost(slice(n - 3, n)),
            "first of a tile": lost(tile), "last of a tile": lost(tile + 63), "tile": lost(slice(tile, tile + 64)),
            "tail": lost(slice(last, n)), "key twice": doubled(tile), "tile twice": doubled(slice(tile, tile + 64)),
            "tile for another": both}


def generator(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


@pytest.mark.parametrize("n", N + [1, 63, 65, 50000])
def test_marks_accept_the_right_result(n):
    values, counts = marks.marked(generator(n), n)
    keys = torch.cat([values, torch.zeros(n, 64)], 1)
    marks.check_marks(*attend(torch.zeros(2, 576), keys, torch.ones(n), 0.072), n, counts)


@pytest.mark.parametrize("n", N + [50000])
@pytest.mark.parametrize("kind", sorted(mistakes(1000)))
def test_marks_refuse(n, kind):
    values, counts = marks.marked(generator(n), n)
    keys = torch.cat([values, torch.zeros(n, 64)], 1)
    wrong = attend(torch.zeros(2, 576), keys, mistakes(n)[kind], 0.072)
    with pytest.raises(AssertionError):
        marks.check_marks(*wrong, n, counts)


def drawn(n):
    g = generator(n + 1)
    keys = torch.randn(n, 576, generator=g).bfloat16()
    return (torch.randn(4, 576, generator=g) / 2).bfloat16(), keys


@pytest.mark.parametrize("n", N)
def test_close_accepts_rounded_weights(n):
    """The kernel's own rounding: weights in bf16 over the sum of those, relative to a whole reference."""
    q, keys = drawn(n)
    s = q.double() @ keys.double().T * (1 / math.sqrt(192.0))
    lse = torch.logsumexp(s, -1)
    y = s / math.log(2.0)
    p = torch.exp2(y - y.amax(-1, keepdim=True).ceil()).bfloat16().double()
    out = (p @ keys[:, :512].double()) / p.sum(-1, keepdim=True)
    marks.check_close(out.bfloat16(), lse.float(), torch.exp(s - lse[:, None]) @ keys[:, :512].double(), lse)


@pytest.mark.parametrize("n", N)
@pytest.mark.parametrize("kind", sorted(mistakes(1000)))
def test_close_refuses(n, kind):
    q, keys = drawn(n)
    scale = 1 / math.sqrt(192.0)
    right, wrong = (attend(q, keys, w, scale) for w in (torch.ones(n), mistakes(n)[kind]))
    s = q.double() @ keys.double().T * scale
    lse = torch.logsumexp(s, -1)
    exact = torch.exp(s - lse[:, None]) @ keys[:, :512].double()
    marks.check_close(*right, exact, lse)
    with pytest.raises(AssertionError):
        marks.check_close(*wrong, exact, lse)
