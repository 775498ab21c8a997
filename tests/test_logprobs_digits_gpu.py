"""Log probabilities keep their own digits: they are as exact as the difference
from the row's maximum and the logarithm of the sum, however large the logits."""
import math

import pytest
import torch

from test_logprobs_gpu import F32_HALF, TYPES, _lib, call, rows  # noqa: F401  (_lib: builds the library)

pytestmark = pytest.mark.gpu


def check(x, k=5):
    """With x - m and ln S apart: one rounding of x - m, one of the difference, two
    of ln S, and the relative error of S (as where sums are tested)."""
    tok = torch.stack([x.float().argmax(1), x.float().argmin(1)], 1).int()
    got = call(x, tok, k)
    d = x.double() - x.double().amax(1, keepdim=True)
    log_s = torch.logsumexp(d, 1, keepdim=True)
    want = d - log_s
    p = want.exp()
    y = (p * d.abs()).sum(1, keepdim=True) / math.log(2) + 1
    rel = (8 + 4 * y + x.shape[1] / 128 + 64) * F32_HALF
    for ids, lp in ((got["ids"], got["top"]), (tok, got["lp"])):
        w = want.gather(1, ids.long().cuda())
        off = (lp.cuda().double() - w).abs()
        tol = rel + 4 * F32_HALF * w.abs()
        assert (off <= tol).all(), float((off / tol).max())
        assert (lp <= 0).all()


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("v", [2, 9, 300, 5000])
@pytest.mark.parametrize("shift", [0, 1000, 20000, -20000, 60000])
def test_shifted_rows(shift, v, dtype):
    for t in (3, 700):
        x, _ = rows(v, t, v, dtype)
        x.add_(shift)
        check(x, min(v, 5))


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("above", [5.0, 15.0, 30.0, 100.0])
def test_confident_rows(above, dtype):
    """One value far above the others: a log probability near 0, never above."""
    for t, v in ((3, 32000), (700, 2000), (2500, 333)):
        x, tok = rows(1, t, v, dtype)
        x.scatter_(1, tok[:, None].long().cuda(), above)
        check(x)
        x.add_(200.0)
        check(x)
