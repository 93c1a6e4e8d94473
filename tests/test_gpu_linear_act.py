"""The linear with an epilogue against the fp64 oracle, within its derived bounds."""

import numpy as np
import pytest
import torch

import mxfp4_block_scaled_quant_amd as mx
from mxfp4_block_scaled_quant_amd import inputs
from oracle import feedforward as D
from oracle import formats as F
from oracle import quant as Q
from tests.helpers import dev_bf16, host_bf16_bits, need_gpu

pytestmark = pytest.mark.gpu


def run(M, N, K, act, gated, bias, residual, seed=0, path=0, out_dtypes=(torch.bfloat16, torch.float32)):
    p = inputs.linear_problem(M, N, K, seed, outliers=True, with_bias=bias)
    cols = N // 2 if gated else N
    r = inputs.activations(M, cols, seed + 9) if residual else None
    W = mx.quantize_weight(dev_bf16(p["w"]))
    ref, err = D.linear_act(p["x"], *Q.quant_1x32(p["w"]), p["bias"], act, gated, r)
    for dt in out_dtypes:
        try:
            mx.set_gemm_path(path)
            y = mx.mxfp4_linear_act(dev_bf16(p["x"]), W.w_pre, W.ws_pre, N, None if p["bias"] is None else dev_bf16(p["bias"]),
                                    act, gated, None if r is None else dev_bf16(r), out_dtype=dt)
        finally:
            mx.set_gemm_path(0)
        assert y.dtype == dt and y.shape == (M, cols)
        if dt == torch.float32:
            got, half = y.double().cpu().numpy(), 2.0 ** -24
        else:
            got, half = F.bf16_to_f64(host_bf16_bits(y)), 2.0 ** -8
        bound = err + half * (np.abs(ref) + err) + 1e-38
        worst = float(np.max(np.abs(got - ref) / bound))
        assert worst <= 1.0, (dt, worst)


FORMS = [("none", False, True, True), ("gelu_tanh", False, True, False), ("silu", True, False, False),
         ("gelu", True, True, True), ("relu", False, False, True)]


@pytest.mark.parametrize("M,N,K", [(1, 32, 32), (1, 1024, 5120), (2, 160, 4128), (3, 96, 512), (4, 4096, 256),
                                   (5, 352, 1056), (16, 1024, 2048), (17, 96, 4128), (37, 96, 4128), (64, 2080, 544),
                                   (65, 4096, 288), (100, 288, 512), (256, 64, 96), (300, 128, 256), (300, 544, 1056),
                                   (513, 1056, 288)])
@pytest.mark.parametrize("act,gated,bias,residual", FORMS)
def test_linear_act(M, N, K, act, gated, bias, residual):
    need_gpu()
    run(M, N, K, act, gated, bias, residual)


@pytest.mark.parametrize("M,N,K", [(1, 97, 64), (3, 50, 96), (40, 133, 128), (90, 261, 160), (300, 515, 96), (257, 36, 128)])
def test_widths_that_are_not_whole_strips(M, N, K):
    need_gpu()
    run(M, N, K, "gelu", False, True, True)
    run(M, N, K, "none", False, False, False)


@pytest.mark.parametrize("path", [1, 2, 3, 4, 5, 6, 7, 8])
@pytest.mark.parametrize("act,gated,bias,residual", FORMS[:4])
def test_every_kernel_form(path, act, gated, bias, residual):
    need_gpu()
    run(48, 1088, 2080, act, gated, bias, residual, path=path)
    if path not in (1, 7, 8):
        run(330, 1120, 1056, act, gated, bias, residual, path=path)


@pytest.mark.parametrize("M", [1, 4, 9, 16, 17, 32, 33, 48, 49, 64])
@pytest.mark.parametrize("path", [0, 7, 8])
def test_row_tiles_of_the_small_kernels(M, path):
    need_gpu()
    run(M, 1088, 5152, "silu", True, True, True, path=path)
    run(M, 1088, 2080, "silu", True, False, False, path=path)
    run(M, 1088, 5152, "gelu", False, True, True, path=path)


def test_gate_of_many_strips():
    """A shape that the persistent form takes without a gate."""
    need_gpu()
    run(64, 12288, 4640, "silu", True, False, False, out_dtypes=(torch.bfloat16,))


def test_without_an_epilogue_it_is_the_linear():
    need_gpu()
    for M, N, K in ((1, 1024, 1024), (3, 96, 512), (40, 224, 512), (300, 544, 512)):
        p = inputs.linear_problem(M, N, K, 1, with_bias=True)
        W = mx.quantize_weight(dev_bf16(p["w"]))
        x, b = dev_bf16(p["x"]), dev_bf16(p["bias"])
        a = mx.mxfp4_linear_act(x, W.w_pre, W.ws_pre, N, b)
        assert torch.equal(a, mx.mxfp4_linear(x, W.w_pre, W.ws_pre, N, b))


@pytest.mark.parametrize("M", [3, 40, 300])
@pytest.mark.parametrize("gated", [False, True])
def test_strides_views_and_in_place(M, gated):
    need_gpu()
    N, K = 192, 160
    cols = N // 2 if gated else N
    p = inputs.linear_problem(M, N, K, 2, with_bias=True)
    W = mx.quantize_weight(dev_bf16(p["w"]))
    x, b, r = dev_bf16(p["x"]), dev_bf16(p["bias"]), dev_bf16(inputs.activations(M, cols, 5))
    ref = mx.mxfp4_linear_act(x, W.w_pre, W.ws_pre, N, b, "silu", gated, r)
    wide = torch.full((M, 400), 3.0, dtype=torch.bfloat16, device="cuda")
    for at, ld in ((0, 400), (8, 400), (2, 400), (6, 400)):
        xs = torch.zeros((M, K + 16), dtype=torch.bfloat16, device="cuda")
        xs[:, 8:8 + K] = x
        res = torch.zeros((M, 301), dtype=torch.bfloat16, device="cuda")
        res[:, 3:3 + cols] = r
        wide.fill_(3.0)
        y = mx.mxfp4_linear_act(xs[:, 8:8 + K], W.w_pre, W.ws_pre, N, b, "silu", gated, res[:, 3:3 + cols],
                                out=wide[:, at:at + cols])
        assert torch.equal(y, ref)
        assert (wide[:, :at] == 3).all() and (wide[:, at + cols:] == 3).all()
        wide[:, at:at + cols] = r
        assert torch.equal(mx.mxfp4_linear_act(x, W.w_pre, W.ws_pre, N, b, "silu", gated, wide[:, at:at + cols],
                                               out=wide[:, at:at + cols]), ref)
        assert (wide[:, :at] == 3).all() and (wide[:, at + cols:] == 3).all()


def test_no_rows():
    need_gpu()
    W = mx.quantize_weight(torch.zeros((64, 32), dtype=torch.bfloat16, device="cuda"))
    x = torch.zeros((0, 32), dtype=torch.bfloat16, device="cuda")
    assert mx.mxfp4_linear_act(x, W.w_pre, W.ws_pre, 64, activation="silu", gated=True).shape == (0, 32)


@pytest.mark.parametrize("M", [2, 37, 320])
def test_captured(M):
    need_gpu()
    N, K = 1024, 1024
    p = inputs.linear_problem(M, N, K, 4)
    W = mx.quantize_weight(dev_bf16(p["w"]))
    x, r = dev_bf16(p["x"]), dev_bf16(inputs.activations(M, N // 2, 6))
    out = torch.zeros_like(r)
    mx.mxfp4_linear_act(x, W.w_pre, W.ws_pre, N, None, "silu", True, r, out=out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mx.mxfp4_linear_act(x, W.w_pre, W.ws_pre, N, None, "silu", True, r, out=out)
    for n in range(3):
        x.copy_(dev_bf16(inputs.activations(M, K, 30 + n)))
        g.replay()
        again = mx.mxfp4_linear_act(x, W.w_pre, W.ws_pre, N, None, "silu", True, r)
        torch.cuda.synchronize()
        assert torch.equal(out, again)


def test_rows_past_32_bits():
    """Outputs and residuals whose last rows lie past 4 GiB, in place."""
    need_gpu()
    M, N, K = 70000, 64, 32
    W = mx.quantize_weight(dev_bf16(inputs.weights(N, K, 3)))
    x = dev_bf16(inputs.activations(M, K, 4))
    r = dev_bf16(inputs.activations(M, N // 2, 5))
    want = mx.mxfp4_linear_act(x, W.w_pre, W.ws_pre, N, None, "silu", True, r)
    wide = torch.empty((M, 40000), dtype=torch.bfloat16, device="cuda")
    at = wide[:, 1024:1024 + N // 2]
    at.copy_(r)
    mx.mxfp4_linear_act(x, W.w_pre, W.ws_pre, N, None, "silu", True, at, out=at)
    assert torch.equal(at, want)
