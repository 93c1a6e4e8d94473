"""Activations over the whole range of their type, in every form of the linear and of the experts' products."""

import math

import numpy as np
import pytest
import torch

import mxfp4_block_scaled_quant_amd as mx
from mxfp4_block_scaled_quant_amd import inputs
from oracle import feedforward as D
from oracle import formats as F
from oracle import quant as Q
from tests.helpers import dev_bf16, need_gpu
from tests.test_gpu_moe import device, problem

pytestmark = pytest.mark.gpu

ACTS = ["none", "silu", "gelu", "gelu_tanh", "relu"]
VALUES = [s * v for v in (0.0, 1.0, 2.0 ** 20, 2.0 ** 63, 1.8e19, 2.0 ** 65, 1e20, 2.0 ** 100, 3e38) for s in (1, -1)]


def _bits(v, n):
    """The values, over and over, as n bf16 numbers."""
    v = np.resize(np.asarray(v, np.float64), n)
    bits = F.f64_to_bf16(np.where(np.isfinite(v), v, 0.0))
    return np.where(np.isfinite(v), bits, np.where(v > 0, 0x7F80, 0xFF80)).astype(np.uint16)


def _linear(M, N, act, gated, values, path, dtype):
    """x = 0 through the linear: the activation (times a factor of 2^-10) of the bias."""
    K = 544
    cols = N // 2 if gated else N
    gate = _bits(values, cols)
    bias = np.concatenate([gate, _bits([2.0 ** -10, -2.0 ** -10, 2.0 ** -10], cols)]) if gated else gate
    W = mx.quantize_weight(dev_bf16(inputs.weights(N, K, 1)))
    try:
        mx.set_gemm_path(path)
        y = mx.mxfp4_linear_act(torch.zeros((M, K), dtype=torch.bfloat16, device="cuda"), W.w_pre, W.ws_pre, N,
                                dev_bf16(bias), act, gated, out_dtype=dtype)
    finally:
        mx.set_gemm_path(0)
    y = y.double().cpu().numpy()
    assert np.array_equal(y, np.repeat(y[:1], M, 0), equal_nan=True)
    return y[0], F.bf16_to_f64(gate), F.bf16_to_f64(bias[cols:]) if gated else np.ones(cols)


# (rows, weight rows, gated too, test path): bf16 rows quantised in the kernel, the small kernels of one to four row
# tiles in both forms, several launches of 64 rows, the large-M kernel at both widths, widths of single elements
FORMS = [(1, 96, True, 0), (3, 96, True, 0), (20, 1088, True, 7), (20, 1088, True, 8), (48, 1088, True, 7),
         (48, 1088, True, 8), (64, 1088, True, 0), (100, 96, True, 3), (330, 1120, True, 2), (330, 1120, True, 4),
         (330, 1120, True, 5), (330, 1120, True, 6), (330, 133, False, 0), (40, 133, False, 0), (2, 133, False, 0)]


@pytest.mark.parametrize("M,N,gates,path", FORMS)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_large_values_of_the_linear(M, N, gates, path, act, dtype):
    need_gpu()
    for gated in (False, True) if gates else (False,):
        y, v, u = _linear(M, N, act, gated, VALUES, path, dtype)
        ref = D.activation(v, act) * u
        # past |v| = 2^20 every activation is v, 0 or within 1e-30 of 0, and the products by 2^-10 are exact: the
        # last rounding of a bf16 value changes nothing; at 1 the power's, the reciprocal's and the products' ulps, at
        # most 8 of 2^-23, and erfc's fit (2.5e-6), before the rounding
        near = np.abs(v) <= 1
        half = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
        bound = np.where(near, (half + 4e-6) * np.abs(ref), 0) + 1e-30
        assert np.isfinite(y).all(), (gated, v[~np.isfinite(y)])
        assert (np.abs(y - ref) <= bound).all(), (gated, v[np.abs(y - ref) > bound])


@pytest.mark.parametrize("M,N,gates,path", FORMS)
@pytest.mark.parametrize("act", ACTS)
def test_infinite_values_of_the_linear(M, N, gates, path, act):
    """+inf stays so; of -inf the formulas leave -inf, 0, or NaN (infinity over infinity, or times 0)."""
    need_gpu()
    for gated in (False, True) if gates else (False,):
        y, v, u = _linear(M, N, act, gated, [math.inf, 1.0, -math.inf, 1.0], path, torch.float32)
        up = v == math.inf
        assert np.array_equal(y[up], u[up] * math.inf), gated
        low = y[v == -math.inf]
        if act == "none":
            assert np.array_equal(low, u[v == -math.inf] * -math.inf)
        elif act == "relu":
            assert (low == 0).all()
        else:
            assert np.isnan(low).all()
        assert np.isfinite(y[v == 1]).all()


# few pairs, one launch's sum, streamed rows, tiles
@pytest.mark.parametrize("T,k,E", [(3, 2, 8), (40, 2, 8), (90, 2, 8), (150, 2, 8)])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("gated", [False, True])
def test_large_values_of_the_experts(T, k, E, act, gated):
    """x = 0: every column of expert e's inner row is act(g_e) (times a power of two that brings it near 1 again), a
    value that E2M1 holds, or 0."""
    need_gpu()
    H, I = 192, 96
    p = problem(T, k, E, H, I, seed=41, gated=gated, bias=True)
    p["x"][:] = 0
    g = np.array([2.0 ** 63, -2.0 ** 63, 2.0 ** 65, -2.0 ** 65, 2.0 ** 100, -2.0 ** 100, 2.0 ** 110, -2.0 ** 110])
    u = 1 / np.abs(g) if gated else np.ones(E)
    p["up_bias"][:, :I] = F.f64_to_bf16(g)[:, None]
    if gated:
        p["up_bias"][:, I:] = F.f64_to_bf16(u)[:, None]
    p["weights"] = (1 + (p["weights"] > 0.5)).astype(np.float32)
    out = mx.mxfp4_moe(**device(p), activation=act, gated=gated).double().cpu().numpy()
    h = np.where((g > 0) | (act == "none"), g, 0) * u
    w = Q.dequant(*p["down"])                                   # [E, H, I]
    y, size = w.sum(2) * h[:, None] + F.bf16_to_f64(p["down_bias"]), np.abs(w).sum(2) * np.abs(h)[:, None]
    ref = sum(p["weights"][:, j, None].astype(np.float64) * y[p["ids"][:, j]] for j in range(k))
    total = sum(p["weights"][:, j, None].astype(np.float64) * (size[p["ids"][:, j]] + np.abs(y[p["ids"][:, j]]))
                for j in range(k))
    # fp32 sums (2^-18 of the terms' magnitudes) and the last rounding
    assert np.isfinite(out).all()
    assert (np.abs(out - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -17 * total).all()
