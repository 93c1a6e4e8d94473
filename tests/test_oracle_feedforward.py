"""The feed-forward oracle against hand-worked and independent forms (CPU)."""

import math

import numpy as np
import torch

from mxfp4_block_scaled_quant_amd import inputs
from oracle import feedforward as D
from oracle import formats as F
from oracle import quant as Q


def test_route_by_hand():
    x = np.array([[0.0, 1.0, 1.0, -np.inf], [-np.inf] * 4, [np.inf, 3.0, np.nan, 2.0]])
    w, ids = D.route(x, 3)
    assert ids.tolist() == [[1, 2, 0], [-1, -1, -1], [0, 1, 3]]
    z = 2 * math.e + 1
    assert np.allclose(w[0], [math.e / z, math.e / z, 1 / z]) and not w[1].any()
    assert w[2].tolist() == [1.0, 0.0, 0.0]
    # the bias chooses, the score weighs
    w, ids = D.route(np.array([[0.0, 2.0]]), 1, np.array([1.0, 0.0]), scoring="sigmoid", renormalize=False, scale=4.0)
    assert ids.tolist() == [[0]] and w.tolist() == [[2.0]]
    # groups of two: sums of two, then of one
    x = np.log(np.array([[0.4, 0.3, 0.5, 0.1]]) / (1 - np.array([[0.4, 0.3, 0.5, 0.1]])))
    assert D.route(x, 1, scoring="sigmoid", groups=2, top_groups=1)[1].tolist() == [[0]]
    assert D.route(x, 1, scoring="sigmoid", groups=2, top_groups=1, group_top=1)[1].tolist() == [[2]]


def test_activations_against_torch():
    v = torch.linspace(-9, 9, 301, dtype=torch.float64)
    for name, f in (("silu", torch.nn.functional.silu), ("relu", torch.relu), ("gelu", torch.nn.functional.gelu),
                    ("gelu_tanh", lambda z: torch.nn.functional.gelu(z, approximate="tanh"))):
        assert np.allclose(D.activation(v.numpy(), name), f(v).numpy(), rtol=1e-12, atol=1e-15)


def test_requantised_contains_the_quantisation_of_values_within_the_bound():
    r = np.random.default_rng(3)
    v = r.standard_normal((6, 128)) * np.exp2(r.integers(-3, 3, (6, 1)))
    err = np.full(v.shape, 2.0 ** -9)
    ref, dev = D.requantised(v, err)
    for _ in range(20):
        z = F.f64_to_bf16(v + err * r.uniform(-1, 1, v.shape))
        assert (np.abs(Q.dequant(*Q.quant_1x32(z)) - ref) <= dev).all()
    same, none = D.requantised(F.bf16_to_f64(F.f64_to_bf16(v)), np.zeros(v.shape))
    assert not none.any() and (same == Q.dequant(*Q.quant_1x32(F.f64_to_bf16(v)))).all()


def test_moe_of_one_expert_is_two_linears():
    x = inputs.activations(5, 64, 1)
    up = Q.quant_1x32(inputs.weights(2 * 96, 64, 1))
    down = Q.quant_1x32(inputs.weights(64, 96, 2))
    ids = np.array([[0, 1], [1, 0], [-1, 7], [0, 0], [1, 2]])
    w = np.arange(10, dtype=float).reshape(5, 2) / 4
    out, err = D.moe(x, ids, w, (up[0][None], up[1][None]), (down[0][None], down[1][None]))
    v, _ = D.linear_act(x, *up, act="silu", gated=True)
    y, _ = D.linear_act(F.f64_to_bf16(v), *down)
    share = np.where(ids == 0, w, 0).sum(1)
    assert np.allclose(out, share[:, None] * y, rtol=1e-12, atol=1e-15) and (err >= 0).all() and not out[2].any()
