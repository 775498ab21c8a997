"""Lengths beyond the table, up to the largest number: the row is cut to what is
wanted and nothing outside it is touched."""
import pytest
import torch

from test_pages_gpu import Model, _lib, fit, same, state  # noqa: F401  (_lib: builds the library)

pytestmark = pytest.mark.gpu
MOST = (1 << 31) - 1


@pytest.mark.parametrize("page", [1, 2, 16])
@pytest.mark.parametrize("want", [0, 1, 30, 40])
@pytest.mark.parametrize("window,sinks", [(0, 0), (5, 3), (MOST, 0)])
@pytest.mark.parametrize("batch", [2, 300, 1100])
def test_lengths_beyond_the_table(batch, want, page, window, sinks):
    width = 40
    m = Model(batch * width + 7, page, batch, width)
    m.rows = [[b * width + c for c in range(width)] for b in range(batch)]
    m.refs = [1] * (batch * width) + [0] * 7
    m.held = [width - b % 2 for b in range(batch)]
    for b in range(1, batch, 2):
        m.refs[m.rows[b][-1]] = 0
        m.rows[b][-1] = -1
    m.lens = [MOST - b % 40 for b in range(batch)]
    table, held, lens, refs = state(m)
    wide = torch.full((batch, width + 64), 123, dtype=torch.int32, device="cuda")
    wide[:, 32:32 + width] = table
    copies, status = fit(m, wide[:, 32:32 + width], held, lens, refs, [want * page] * batch, window, sinks)
    assert status == 0 and copies == [list(c) for c in m.fit([want * page] * batch, window, sinks)]
    same(m, wide[:, 32:32 + width], held, refs)
    assert (wide[:, :32] == 123).all() and (wide[:, 32 + width:] == 123).all()
