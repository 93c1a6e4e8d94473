"""The choice of groups where fp32 scores cannot tell them apart: cancelling biases, near ties, masks of the lowest value."""

import numpy as np
import pytest
import torch

import mxfp4_block_scaled_quant_amd as mx
from oracle import feedforward as D
from tests.helpers import need_gpu

pytestmark = pytest.mark.gpu

LOWEST = float(np.finfo(np.float32).min)


def _scores64(x, b, scoring):
    x = x.astype(np.float64)
    there = (x > -np.inf) & (b > -np.inf)
    s = 1 / (1 + np.exp(-x))
    if scoring == "softmax":
        s = np.exp(np.where(there, x, -np.inf) - np.where(there, x, -np.inf).max(1, keepdims=True))
        s = s / s.sum(1, keepdims=True)
    return np.where(there, s + b, -np.inf)


def _group_scores(c, groups, group_top):
    top = np.sort(c.reshape(len(c), groups, -1), 2)[:, :, ::-1][:, :, :group_top]
    return np.where(top > -np.inf, top, 0).sum(2)


def _same_choice(x, b, k, scoring, groups, keep, group_top):
    """ids equal the 64-bit choice, but where the scores that decide are themselves a rounding of 64 bits apart."""
    kw = dict(scoring=scoring, groups=groups, top_groups=keep, group_top=group_top)
    ids = mx.moe_route(torch.from_numpy(x).cuda(), k, torch.from_numpy(b).cuda(), **kw)[1].cpu().numpy()
    n = min(len(x), 300)
    ref = D.route(x[:n].astype(np.float64), k, b.astype(np.float64), **kw)[1]
    differ = np.nonzero((ids[:n] != ref).any(1))[0]
    size = x.shape[1] // groups
    for t in differ:
        c = _scores64(x[t:t + 1], b.astype(np.float64), scoring)
        near = 2.0 ** -50 * (1 + np.abs(b[np.isfinite(b)]).max())
        g = _group_scores(c, groups, group_top)[0]
        kept, want = (sorted(set((z[z >= 0] // size).tolist())) for z in (ids[t], ref[t]))
        assert len(kept) == len(want) and np.allclose(g[kept], g[want], rtol=0, atol=near), (t, ids[t], ref[t])
        assert np.allclose(c[0][ids[t]], c[0][ref[t]], rtol=0, atol=near), (t, ids[t], ref[t])
    assert len(differ) <= n // 50
    return ids


# the three kernels, each with groups that fill lanes and (the first) with groups that do not
SHAPES = [(70, 4, 2), (70, 64, 8), (70, 60, 6), (70, 256, 8), (70, 256, 16), (70, 200, 25), (70, 1024, 32),
          (8200, 128, 8), (8200, 256, 16)]


@pytest.mark.parametrize("T,E,groups", SHAPES)
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("large", [8.0, 64.0, 1000.0, 1e5])
def test_biases_that_cancel(T, E, groups, scoring, large):
    """A group's two scores are s + B and s - B: their fp32 roundings, of B's size, stay in a sum of theirs that is
    small, and the groups' sums are nearer than that."""
    need_gpu()
    r = np.random.default_rng([3, T, E])
    size = E // groups
    x = np.full((T, groups, size), -9.0, np.float32)
    x[:, :, :2] = r.standard_normal((T, 1, 2))
    x += (r.integers(-40, 41, x.shape) * 2.0 ** -23).astype(np.float32)
    b = np.full((groups, size), -4 * large, np.float32)
    b[:, 0], b[:, 1] = large, -large
    for keep in (1, groups // 2):
        _same_choice(x.reshape(T, E), b.reshape(E), 2, scoring, groups, keep, 2)


@pytest.mark.parametrize("T", [64, 8200])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group_top", [1, 2])
def test_groups_whose_scores_are_less_than_an_ulp_apart(T, scoring, group_top):
    need_gpu()
    r = np.random.default_rng(6)
    base = r.standard_normal((T, 1)).astype(np.float32)
    x = (base + r.integers(-3, 4, (T, 128)).astype(np.float32) * np.float32(2.0 ** -24)).astype(np.float32)
    for b in ((r.integers(-2, 3, 128) * 2.0 ** -26).astype(np.float32), np.full(128, 0.25, np.float32)):
        for groups, keep in ((8, 2), (16, 5)):
            _same_choice(x, b, 8, scoring, groups, keep, group_top)


@pytest.mark.parametrize("T,E,groups", [(40, 64, 8), (40, 60, 6), (40, 128, 16), (40, 256, 16), (8200, 128, 16)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group_top", [1, 2])
def test_masks_of_the_lowest_value(T, E, groups, scoring, group_top):
    """A bias of the type's lowest value is not -inf: its expert comes last, and two of them, whose sum is past fp32,
    leave their group in the choice."""
    need_gpu()
    r = np.random.default_rng([9, E])
    size = E // groups
    x = r.standard_normal((T, E)).astype(np.float32)
    b = np.full((groups, size), LOWEST, np.float32)
    b[1], b[4] = 0, -np.inf                     # one group is open, one closed
    assert (_same_choice(x, b.reshape(E), size + 1, scoring, groups, 2, group_top) >= 0).all()
    b[3, 2] = 0.5                               # and one of a single expert
    assert (_same_choice(x, b.reshape(E), size + 1, scoring, groups, 3, group_top) >= 0).all()
    x[:, :size * 2] = LOWEST                    # and logits of it
    _same_choice(x, b.reshape(E), size + 1, scoring, groups, 3, group_top)
