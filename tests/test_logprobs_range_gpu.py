"""Log probabilities of rows far from 0, where a value's exponent rounds by more
than the exponent that is left of it beside the row's maximum."""
import pytest
import torch

from test_logprobs_gpu import TYPES, _lib, check, rows  # noqa: F401  (_lib: builds the library)

pytestmark = pytest.mark.gpu

# The second and third leave a maximum of an exponent between -128 and -126, whose
# power of two is no normal number, to a product rounded once.
FAR = [1e6, 3184999936.0, 3159000064.0, 1.1e6, 999999.0, 1e7, 1e9, 1e10, 1e20, 1e30, 0.9e38]
WIDE = [torch.bfloat16, torch.float32]
PATTERNS = {
    "all equal": lambda x, v: x.fill_(v),
    "one": lambda x, v: x[:, x.shape[1] // 2].fill_(v),
    "every 17th": lambda x, v: x[:, 3::17].fill_(v),
    "half": lambda x, v: (x.fill_(-v), x[:, ::2].fill_(v)),
    "around": lambda x, v: x.add_(v),
}


@pytest.mark.parametrize("dtype", WIDE, ids=str)
@pytest.mark.parametrize("v", [8, 13, 300, 40000])
@pytest.mark.parametrize("far", [s * f for f in FAR for s in (1, -1)])
def test_far_rows(far, v, dtype):
    for t in (2, 700):
        for pattern in PATTERNS.values():
            x, tok = rows(7, t, v, dtype)
            pattern(x, far)
            check(x, tok, min(v, 5))


@pytest.mark.parametrize("low", [-64000.0, -64992.0, -65024.0, -65400.0, 65504.0])
def test_far_half_rows(low):
    """The ends of fp16's range, whose neighbours are 32 apart."""
    for t in (2, 700):
        for pattern in PATTERNS.values():
            x, tok = rows(8, t, 3000, torch.float16)
            pattern(x, low)
            x.clamp_(-65504, 65504)
            check(x, tok, 5)
