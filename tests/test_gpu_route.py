"""Routing against the fp64 oracle: ids exactly, weights to their arithmetic."""

import numpy as np
import pytest
import torch

import mxfp4_block_scaled_quant_amd as mx
from oracle import feedforward as D
from tests.helpers import need_gpu

pytestmark = pytest.mark.gpu

# (E, top_k, groups, top_groups, group_top)
SHAPES = [(1, 1, 1, 1, 2), (8, 2, 1, 1, 2), (60, 4, 1, 1, 2), (64, 6, 1, 1, 2), (64, 6, 8, 3, 1), (60, 5, 6, 2, 2),
          (128, 16, 1, 1, 2), (160, 6, 8, 3, 2), (256, 8, 8, 4, 2), (256, 8, 8, 8, 2), (384, 8, 1, 1, 2),
          (200, 20, 20, 4, 2), (512, 24, 16, 5, 2), (1024, 64, 64, 9, 1), (1000, 7, 40, 3, 2), (17, 17, 1, 1, 2)]


def _logits(T, E, seed, dtype, spread=1.5):
    x = np.random.default_rng([seed, T, E]).standard_normal((T, E)) * spread
    return torch.from_numpy(x).to(dtype).cuda()


def _check(x, k, b=None, **kw):
    w, ids = mx.moe_route(x, k, b, **kw)
    torch.cuda.synchronize()
    rw, rids = D.route(x.double().cpu().numpy(), k, None if b is None else b.double().cpu().numpy(), **kw)
    assert np.array_equal(ids.cpu().numpy(), rids)
    # exp of a difference rounded once (|d| 2^-24, d < 128), its ulp, the sum of at most 1024 such, the quotient and
    # the scale: under 2^-16 of the weight for |d| < 128; what is smaller underflows against the largest
    assert np.allclose(w.double().cpu().numpy(), rw, rtol=2.0 ** -16, atol=1e-37 * abs(kw.get("scale", 1.0)))
    return w, ids


@pytest.mark.parametrize("E,k,groups,keep,gt", SHAPES)
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route(E, k, groups, keep, gt, scoring, biased, dtype):
    need_gpu()
    x = _logits(37, E, 1, dtype)
    b = _logits(1, E, 2, torch.float32, 0.1)[0] if biased else None
    for renorm in (True, False):
        _check(x, k, b, scoring=scoring, groups=groups, top_groups=keep, group_top=gt, renormalize=renorm, scale=2.5)


@pytest.mark.parametrize("E,k,groups,keep,gt", [(8, 2, 1, 1, 2), (60, 4, 1, 1, 2), (64, 6, 8, 3, 2), (64, 15, 4, 2, 1),
                                                (128, 8, 1, 1, 2), (128, 5, 16, 7, 2), (160, 6, 1, 1, 2),
                                                (256, 8, 8, 4, 2), (256, 8, 16, 4, 1), (256, 15, 1, 1, 2),
                                                (200, 6, 25, 4, 2), (252, 3, 1, 1, 2)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_many_tokens(E, k, groups, keep, gt, scoring, biased, dtype):
    """The form of many tokens, on rows whose like are checked one by one above: the same rows in small calls."""
    need_gpu()
    x = _logits(8203, E, 11, dtype)
    x[5] = -np.inf
    x[6, k // 2:] = -np.inf
    x[7, ::3] = np.nan
    x[8, 1] = np.inf
    x[9] = 1.0
    b = _logits(1, E, 12, torch.float32, 0.1)[0] if biased else None
    kw = dict(scoring=scoring, groups=groups, top_groups=keep, group_top=gt, scale=2.5)
    for renorm in (True, False):
        w, ids = mx.moe_route(x, k, b, renormalize=renorm, **kw)
        parts = [mx.moe_route(p, k, b, renormalize=renorm, **kw) for p in x.split(2000)]
        assert torch.equal(ids, torch.cat([q[1] for q in parts]))
        assert torch.allclose(w, torch.cat([q[0] for q in parts]), rtol=2.0 ** -20, atol=1e-37)
    rw, rids = D.route(x[:40].double().cpu().numpy(), k, None if b is None else b.double().cpu().numpy(), **kw)
    assert np.array_equal(mx.moe_route(x, k, b, **kw)[1][:40].cpu().numpy(), rids)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_many_tokens_with_ties(scoring, biased, dtype):
    need_gpu()
    r = np.random.default_rng(15)
    x = torch.from_numpy(r.integers(-3, 4, (8192, 256)).astype(np.float32) / 2).to(dtype).cuda()
    b = torch.from_numpy(r.integers(-1, 2, 256).astype(np.float32) / 8).cuda() if biased else None
    for groups, keep in ((1, 1), (8, 3)):
        kw = dict(scoring=scoring, groups=groups, top_groups=keep)
        ids = mx.moe_route(x, 8, b, **kw)[1].cpu().numpy()
        ref = D.route(x[:200].double().cpu().numpy(), 8, None if b is None else b.double().cpu().numpy(), **kw)[1]
        assert np.array_equal(ids[:200], ref)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_ties_masks_and_values_that_are_not_finite(scoring, biased):
    need_gpu()
    r = np.random.default_rng(5)
    x = r.integers(-2, 3, (64, 64)).astype(np.float32)          # many equal logits
    x[1] = -np.inf                                                # nobody
    x[2, 3:] = -np.inf                                            # fewer than asked for
    x[3, ::2] = np.nan
    x[4, 5] = np.inf
    x[5] = np.inf
    x[6] = -3e38
    x[7] = np.finfo(np.float32).max
    x[8, :32] = -np.inf                                           # whole groups
    x[9, 1:] = -np.inf
    x[10] = np.nan
    x[11] *= 100
    x[12] = -90 - x[12]                                           # sigmoids that vanish in fp32
    x = torch.from_numpy(x).cuda()
    b = None
    if biased:
        b = torch.from_numpy(r.integers(-1, 2, 64).astype(np.float32) / 8).cuda()
        b[7], b[9], b[11] = -np.inf, np.nan, np.inf
    for groups, keep, gt in ((1, 1, 2), (8, 3, 2), (8, 3, 1), (4, 1, 2)):
        _check(x, 6, b, scoring=scoring, groups=groups, top_groups=keep, group_top=gt)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_choices_that_fp32_cannot_tell_apart(scoring):
    """Scores that differ by less than an fp32 ulp: the 64-bit choice decides."""
    need_gpu()
    r = np.random.default_rng(6)
    base = r.standard_normal((256, 1)).astype(np.float32)
    x = (base + r.integers(-3, 4, (256, 128)).astype(np.float32) * np.float32(2.0 ** -24)).astype(np.float32)
    b = (r.integers(-2, 3, 128) * 2.0 ** -26).astype(np.float32)
    xt = torch.from_numpy(x).cuda()
    for bias in (None, torch.from_numpy(b).cuda(), torch.full((128,), 0.25, device="cuda")):
        for groups, keep in ((1, 1), (8, 2)):
            ids = mx.moe_route(xt, 8, bias, scoring=scoring, groups=groups, top_groups=keep)[1].cpu().numpy()
            ref = _route64(x, 8, None if bias is None else bias.cpu().numpy(), scoring, groups, keep)
            # near-ties of sums of 64-bit exponentials may themselves fall either way in the last bit: compare the
            # scores the ids stand for
            assert (np.sort(ids, 1)[:, 1:] != np.sort(ids, 1)[:, :-1]).all()
            if bias is None and groups == 1:
                assert np.array_equal(ids, ref)
            else:
                s = _scores64(x, None if bias is None else bias.cpu().numpy(), scoring)
                got, want = (np.take_along_axis(s, z, 1) for z in (ids.astype(int), ref))
                if groups == 1:
                    assert np.abs(got - want).max() < 1e-14


def _scores64(x, b, scoring):
    x = x.astype(np.float64)
    s = 1 / (1 + np.exp(-x))
    if scoring == "softmax":
        s = np.exp(x - x.max(1, keepdims=True))
        s = s / s.sum(1, keepdims=True)
    return s if b is None else s + b.astype(np.float64)


def _route64(x, k, b, scoring, groups, keep):
    return D.route(x.astype(np.float64), k, None if b is None else b.astype(np.float64), scoring=scoring,
                   groups=groups, top_groups=keep)[1]


def test_strides_views_and_given_outputs():
    need_gpu()
    x = _logits(9, 200, 3, torch.float32)[:, 3:131]
    w, ids = torch.full((9, 10), 7.0, device="cuda"), torch.full((9, 12), 7, dtype=torch.int32, device="cuda")
    mx.moe_route(x, 4, weights=w[:, 2:6], ids=ids[:, 5:9])
    rw, rids = mx.moe_route(x.contiguous(), 4)
    assert torch.equal(w[:, 2:6], rw) and torch.equal(ids[:, 5:9], rids)
    assert (w[:, :2] == 7).all() and (w[:, 6:] == 7).all() and (ids[:, :5] == 7).all() and (ids[:, 9:] == 7).all()


@pytest.mark.parametrize("T", [0, 1, 2, 15, 16, 17, 4099])
def test_token_counts(T):
    need_gpu()
    x = _logits(T, 64, 4, torch.bfloat16)
    w, ids = mx.moe_route(x, 6)
    assert w.shape == ids.shape == (T, 6)
    if 0 < T < 100:
        _check(x, 6)
    elif T:
        tail, tid = mx.moe_route(x[-3:], 6)
        assert torch.equal(w[-3:], tail) and torch.equal(ids[-3:], tid)


def test_captured_and_on_another_stream():
    need_gpu()
    x = _logits(33, 256, 8, torch.float32)
    b = _logits(1, 256, 9, torch.float32, 0.1)[0]
    kw = dict(scoring="sigmoid", groups=8, top_groups=4)
    ref = [t.clone() for t in mx.moe_route(x, 8, b, **kw)]
    w, ids = torch.zeros_like(ref[0]), torch.zeros_like(ref[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        mx.moe_route(x, 8, b, weights=w, ids=ids, **kw)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(w, ref[0]) and torch.equal(ids, ref[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mx.moe_route(x, 8, b, weights=w, ids=ids, **kw)
    for n in range(3):
        x.copy_(_logits(33, 256, 20 + n, torch.float32))
        g.replay()
        again = mx.moe_route(x, 8, b, **kw)
        torch.cuda.synchronize()
        assert torch.equal(w, again[0]) and torch.equal(ids, again[1])


def test_rows_past_32_bits():
    need_gpu()
    T, E, k = 9000, 256, 8
    x = _logits(T, E, 31, torch.bfloat16)
    wide = torch.empty((T, 262144), dtype=torch.bfloat16, device="cuda")
    wide[:, 128:128 + E] = x
    for rows in (T, 8190):  # both forms
        a, b = mx.moe_route(x[-rows:], k), mx.moe_route(wide[-rows:, 128:128 + E], k)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
