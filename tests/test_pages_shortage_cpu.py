"""Refusals of the fit that says which lengths may be written to."""
import pytest

import __graft_entry__
from speculative_decode_mla_tree_gb300 import abi

from test_around_cpu import CALLS, FAKE, REFUSED


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build_library()
    return abi.load()


def call(lib, **kw):
    a = {**CALLS["mla_pages_fit"], "step": 2 * FAKE, **kw}
    step = a.pop("step")
    names = list(a)
    v = [a[n] for n in names]
    v.insert(names.index("copies") + 1, step)
    return lib.mla_pages_fit_lens(*v)


@pytest.mark.parametrize("kw", REFUSED["mla_pages_fit"] + [dict(step=FAKE), dict(step=FAKE + 4), dict(step=FAKE - 4),
                                                           dict(lens=2 * FAKE), dict(want=2 * FAKE - 4), dict(held=2 * FAKE + 4)],
                         ids=str)
def test_refuses(lib, kw):
    assert call(lib, **kw) == abi.MT_EINVAL


def test_limits(lib):
    assert call(lib, batch=65536, step=1 << 40) == abi.MT_EUNSUPPORTED
    assert call(lib, ws_bytes=8) == abi.MT_EWORKSPACE and call(lib, ws=None, step=None) == abi.MT_EWORKSPACE
    assert call(lib, batch=0, step=FAKE) == abi.MT_OK
