"""Strided views and a residual in place in every form of the experts' products."""

import pytest
import torch

import mxfp4_block_scaled_quant_amd as mx
from tests.helpers import need_gpu
from tests.test_gpu_moe import check, device, problem

pytestmark = pytest.mark.gpu


def _view(t, before, after):
    """t as a view of wider rows, whose other columns hold a number that must stay."""
    wide = torch.full((t.shape[0], before + t.shape[1] + after), 3, dtype=t.dtype, device=t.device)
    at = wide[:, before:before + t.shape[1]]
    at.copy_(t)
    return wide, at


# few pairs, one launch's sum, streamed rows, tiles
@pytest.mark.parametrize("T,k,E", [(3, 2, 4), (40, 2, 16), (70, 4, 16), (170, 5, 16)])
@pytest.mark.parametrize("hidden", [96, 288])
def test_views_and_in_place(T, k, E, hidden):
    need_gpu()
    p = problem(T, k, E, hidden, 160, seed=51, residual=True, bias=True, elsewhere=True)
    d = device(p)
    want = mx.mxfp4_moe(**d)
    check(p, want)
    wide = {}
    for name, before, after in (("x", 8, 16), ("residual", 12, 4), ("ids", 3, 2), ("weights", 1, 1)):
        wide[name], d[name] = _view(d[name], before, after)
    full, out = _view(torch.zeros_like(want), 4, 8)
    assert torch.equal(mx.mxfp4_moe(**d, out=out), want)
    assert torch.equal(mx.mxfp4_moe(**d, out=d["residual"]), want)
    for t, before, width in ((full, 4, hidden), (wide["x"], 8, hidden), (wide["residual"], 12, hidden), (wide["ids"], 3, k),
                             (wide["weights"], 1, k)):
        assert (t[:, :before] == 3).all() and (t[:, before + width:] == 3).all()
