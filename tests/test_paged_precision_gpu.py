"""How far a decode result may move with what should not matter: the rest of
the batch, and the rounding of the weights for the product with the values."""
import math

import pytest
import torch

import __graft_entry__

import paged_ref as ref
from test_paged_gpu import BF, decode, gen, normal, paged

pytestmark = pytest.mark.gpu

LAYOUTS = pytest.mark.parametrize("page,gap", [(64, 0), (5, 0), (5, 8)], ids=["boxes", "rows", "any"])
# Scores in log2 are this scale times log2 e, in fp32 exactly 1, times q . k
LOG2 = float(torch.tensor(math.log(2.0)))


@pytest.fixture(scope="module", autouse=True)
def _lib():
    __graft_entry__.build()


def test_scale_is_one_in_log2():
    assert float(torch.tensor(LOG2) * torch.tensor(1.4426950408889634)) == 1.0


def eighths(g, std, *shape):
    return (torch.randn(*shape, generator=g) * std * 8).round() / 8


@LAYOUTS
@pytest.mark.parametrize("heads", [16, 24, 64])
def test_decode_alone_as_in_any_batch(heads, page, gap):
    """One request alone and inside batches, where shares end elsewhere. Scores
    are whole 64ths in log2, so they and their distances are exact, and only the
    order of fp32 sums may differ: 4096 keys are 256 steps of 16 keys (and fewer
    than 64 partials), each off by at most 2^-23 of the running sum, on both
    sides 2 x 320 x 2^-23 = 7.7e-5 of an output; a bf16 step is 2^-8 of it at
    least, so at most 2% of the outputs may round the other way (5% allowed),
    and by one step. A weight rounded relative to another reference would move
    outputs by 1.4e-3 and more than a third of them to another value."""
    g = gen(60 + heads)
    n = 4096
    others = [[], [700, 33], [64] * 60, [4096, 1], [0, 5000, 0], [30] * 400]
    one = torch.cat([normal(g, n, 512), eighths(g, 1.0, n, 64).to(BF)], 1)
    qone = torch.cat([torch.zeros(heads, 512), eighths(g, 0.25, heads, 64)], 1).to(BF)
    results = []
    for k, lens in enumerate(others):
        lens = lens + [n] + ([90, 2000] if k % 2 else [])
        at = len(others[k])
        cache, flat, table = paged(g, lens, page, gap=gap)
        flat[ref.slots_of(table[at], page, 0, n)] = one
        cache.copy_(flat.view(cache.shape))
        q = normal(g, len(lens), heads, 576)
        q[at] = qone
        out, lse = decode(q.cuda(), cache, table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"),
                          scale=LOG2)
        results.append((out[at].double().cpu(), lse[at].double().cpu()))
    s = qone.double() @ one.double().T * math.log(2.0)
    exact = torch.logsumexp(s, -1)
    weight = torch.exp(s - exact[:, None]) @ one[:, :512].double().abs()
    for out, lse in results:
        # sums of at most 128 + 16 weights in a row a thread, exp2 and log2 to two units in the last place
        assert ((lse - exact).abs() <= 160 * ref.F32_HALF * 2 + exact.abs() * 8 * ref.F32_HALF).all()
        a, b = results[0][0], out
        step = 2 * ref.BF16_HALF * torch.maximum(a.abs(), b.abs())
        assert ((a - b).abs() <= step + 640 * 2 * ref.F32_HALF * weight).all()
        assert (a != b).double().mean() <= 0.05, (a != b).double().mean()


@LAYOUTS
@pytest.mark.parametrize("lens", [[65] * 320, [129, 1, 640] * 110, [20011], [2560] * 60],
                         ids=["two_tiles", "ragged", "long", "batch"])
def test_decode_average_of_equal_values_is_the_value(lens, page, gap):
    """All values of a request alike: whatever the weights and however they are
    rounded, their average is that value, to the few steps of fp32 in which the
    sums of both sides differ (2^-13 for 20011 keys, under half a step of bf16,
    2^-9). Every second tile begins with a key at 0, the next one ends with one
    at 7 to 8 in log2, the rest are far below: within a share that holds both,
    the larger weight is up to 2^8 and rarely a bf16 value."""
    g = gen(70)
    heads = 64
    cache, flat, table = paged(g, lens, page, gap=gap)
    value = normal(g, len(lens), 512)
    q = torch.zeros(len(lens), heads, 576)
    q[:, :, 512] = 1.0
    q[:, :, 513] = torch.arange(heads) / 64.0
    for b, n in enumerate(lens):
        rows = ref.slots_of(table[b], page, 0, n)
        late = torch.cat([rows[127::128], rows[-1:]])
        flat[rows, :512] = value[b]
        flat[rows, 512:] = 0.0
        flat[rows, 512] = -100.0
        flat[rows[::128], 512] = 0.0
        flat[late, 512] = 7.0
        flat[late, 513] = 1.0
    cache.copy_(flat.view(cache.shape))
    out, lse = decode(q.to(BF).cuda(), cache, table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"),
                      scale=LOG2)
    assert torch.equal(out.cpu(), value[:, None].expand(-1, heads, -1))
    for b in sorted(set(lens.index(n) for n in lens)):
        keys = flat[ref.slots_of(table[b], page, 0, lens[b]), 512:].double()
        want = torch.logsumexp(q[b, :, 512:].double() @ keys.T * math.log(2.0), -1)
        # sums of at most 128 + 16 weights in a row a thread, exp2 and log2 to two units in the last place
        assert ((lse[b].double().cpu() - want).abs() <= 160 * 2 * ref.F32_HALF + want.abs() * 8 * ref.F32_HALF).all()
