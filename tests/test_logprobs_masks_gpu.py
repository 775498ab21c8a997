"""Rows whose masked places hold a number instead of -inf: what is masked has
weight 0 either way, so the sums are the same to the last bit, which those that
are taken again value by value would not be."""
import math

import pytest
import torch

from test_logprobs_gpu import TYPES, _lib, call, check, rows  # noqa: F401  (_lib: builds the library)

pytestmark = pytest.mark.gpu
FILLS = {torch.bfloat16: [-1e5, -2e6, -1e9, -1e10, -1e20, -1e30, -3.3895e38],
         torch.float32: [-1e5, -2e6, -1e9, -1e10, -1e20, -1e30, -3.4028234e38],
         torch.float16: [-3e4, -65504.0]}


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("t,v", [(1, 40000), (3, 8192), (40, 3001), (700, 40000), (1500, 2000)])
def test_any_fill_is_a_mask(t, v, dtype):
    for left in (3, v // 100, v // 3):
        x, tok = rows(left, t, v, dtype, shift=3)
        g = torch.Generator(device="cuda")
        g.manual_seed(left)
        keep = torch.rand(t, v, generator=g, device="cuda").argsort(dim=1)[:, :left]  # some in each row
        hide = torch.ones(t, v, dtype=torch.bool, device="cuda").scatter_(1, keep, False)
        tok = keep[:, 0].int().cpu()
        x.masked_fill_(hide, -math.inf)
        want = call(x, tok, 3)
        for fill in FILLS[dtype]:
            x.masked_fill_(hide, fill)
            got = call(x, tok, 3)
            assert all(torch.equal(got[n], want[n]) for n in want), (fill, left)
            check(x, tok, min(v, 8))
