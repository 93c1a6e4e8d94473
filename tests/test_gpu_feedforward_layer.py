"""Routing, experts and the linears with an epilogue run together, as a layer uses them."""

import importlib.util
import os

import numpy as np
import pytest
import torch

import mxfp4_block_scaled_quant_amd as mx
from mxfp4_block_scaled_quant_amd import inputs, ops  # noqa: F401
from oracle import feedforward as D
from oracle import formats as F
from oracle import quant as Q
from tests.helpers import dev_bf16, host_bf16_bits, need_gpu

pytestmark = pytest.mark.gpu

E, K, HIDDEN, INNER = 16, 4, 256, 128
ROUTE = dict(scoring="sigmoid", groups=4, top_groups=2, scale=2.5)


def _example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "mixture_of_experts.py")
    spec = importlib.util.spec_from_file_location("mixture_of_experts", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    return ex


def _weights():
    up = Q.quant_1x32(inputs.weights(E * 2 * INNER, HIDDEN, 1).reshape(E, 2 * INNER, HIDDEN))
    down = Q.quant_1x32(inputs.weights(E * HIDDEN, INNER, 2).reshape(E, HIDDEN, INNER))
    sup, sdown = inputs.weights(2 * INNER, HIDDEN, 3), inputs.weights(HIDDEN, INNER, 4)
    place = lambda q, s: mx.MXFP4Weight(  # noqa: E731
        *mx.mxfp4_preshuffle_weight(torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda(), q.shape[1],
                                    2 * q.shape[2], batch=E), q.shape[1], 2 * q.shape[2], E)
    dev = (place(*up), place(*down), mx.quantize_weight(dev_bf16(sup)), mx.quantize_weight(dev_bf16(sdown)))
    return dev, (up, down, Q.quant_1x32(sup), Q.quant_1x32(sdown))


def _layer(x, logits, bias, dev):
    up, down, sup, sdown = dev
    w, ids = mx.moe_route(logits, K, bias, **ROUTE)
    y = mx.mxfp4_moe(x, ids, w, up, down, residual=x)
    h = mx.mxfp4_linear_act(x, sup.w_pre, sup.ws_pre, sup.N, activation="silu", gated=True)
    out = mx.mxfp4_linear_act(h, sdown.w_pre, sdown.ws_pre, sdown.N, residual=y)
    return w, ids, y, h, out


def _near(t, ref, err):
    got = F.bf16_to_f64(host_bf16_bits(t))
    bound = err + 2.0 ** -8 * (np.abs(ref) + err) + 1e-38
    worst = float(np.max(np.abs(got - ref) / bound))
    assert worst <= 1.0, worst


@pytest.mark.parametrize("T", [1, 3, 64, 200])
def test_layer_step_by_step(T):
    """Each step against the oracle on what the step before wrote."""
    need_gpu()
    dev, host = _weights()
    x = inputs.activations(T, HIDDEN, 5, outliers=True)
    r = np.random.default_rng(6)
    logits, bias = r.normal(0, 1.5, (T, E)).astype(np.float32), r.normal(0, 0.1, E).astype(np.float32)
    w, ids, y, h, out = _layer(dev_bf16(x), torch.from_numpy(logits).cuda(), torch.from_numpy(bias).cuda(), dev)
    rw, rids = D.route(logits.astype(np.float64), K, bias.astype(np.float64), **ROUTE)
    assert np.array_equal(ids.cpu().numpy(), rids)
    w = w.double().cpu().numpy()
    # a sigmoid, the sum of K of them, a quotient and the scale, in fp32: a dozen roundings
    assert np.all(np.abs(w - rw) <= 12 * 2.0 ** -24 * rw)
    _near(y, *D.moe(x, rids, w, host[0], host[1], residual_bf16=x, half=T * K > 24 * E))
    _near(h, *D.linear_act(x, *host[2], None, "silu", True))
    _near(out, *D.linear_act(host_bf16_bits(h), *host[3], None, residual_bf16=host_bf16_bits(y)))


@pytest.mark.parametrize("T", [1, 24, 320])
def test_layer_captured(T):
    """One graph of the whole layer, replayed over changing tokens between eager calls."""
    need_gpu()
    dev, _ = _weights()
    bias = torch.linspace(-0.1, 0.1, E, device="cuda")
    x, logits = torch.zeros((T, HIDDEN), dtype=torch.bfloat16, device="cuda"), torch.zeros((T, E), device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        _layer(x, logits, bias, dev)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = _layer(x, logits, bias, dev)
    for n in range(4):
        x.copy_(dev_bf16(inputs.activations(T, HIDDEN, 70 + n)))
        logits.copy_(torch.from_numpy(np.random.default_rng(n).normal(0, 2, (T, E)).astype(np.float32)).cuda())
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, _layer(x, logits, bias, dev)):
            assert torch.equal(a, b)


def test_custom_ops_are_the_binding():
    need_gpu()
    (up, down, sup, sdown), _ = _weights()
    x, logits = dev_bf16(inputs.activations(33, HIDDEN, 8)), torch.linspace(-2, 2, 33 * E, device="cuda").reshape(33, E)
    bias = torch.linspace(0.1, -0.1, E, device="cuda")
    w, ids = mx.moe_route(logits, K, bias, **ROUTE)
    cases = [
        (torch.ops.mxfp4.moe_route.default, (logits, K, bias, "sigmoid", 4, 2, 2, True, 2.5), (w, ids)),
        (torch.ops.mxfp4.moe.default, (x, ids, w, up.w_pre, up.ws_pre, down.w_pre, down.ws_pre, E, INNER, None, None,
                                       "silu", True, x), (mx.mxfp4_moe(x, ids, w, up, down, residual=x),)),
        (torch.ops.mxfp4.linear_act.default, (x, sup.w_pre, sup.ws_pre, sup.N, None, "gelu", True),
         (mx.mxfp4_linear_act(x, sup.w_pre, sup.ws_pre, sup.N, activation="gelu", gated=True),)),
    ]
    for op, args, want in cases:
        torch.library.opcheck(op, args, test_utils=("test_schema", "test_faketensor", "test_aot_dispatch_dynamic"))
        got = op(*args)
        for a, b in zip(got if isinstance(got, tuple) else (got,), want):
            assert torch.equal(a, b)


def test_example_in_shards():
    need_gpu()
    # The layer rounds its routed part once to bf16 and its output once; the
    # shards round each their part (two), their sum and the output: six half
    # steps of 2^-8 of the largest value on the way, and two more for the rows
    # of many tokens, held in fp16 before they are weighted (2^-11 each).
    for tokens in (1, 40, 200):
        off, top = _example().demo(tokens=tokens, hidden=512, inner=256, experts=16)
        assert np.isfinite(top) and off <= 8 * 2.0 ** -8 * top
