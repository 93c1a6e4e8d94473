"""Routing, the experts' products and the linear's epilogue, in fp64 from their
definitions (test infrastructure only).

Inputs are bf16 bit patterns (uint16 arrays) for tensors that the library
takes in bf16, packed MXFP4 as :mod:`oracle.quant` makes it, fp64 otherwise.
The products also return the tolerance that a kernel with fp32 sums is held
to: 2^-18 of sum |a b| (plus |bias|) before the activation, carried through
the activation's slope, and for the experts through the quantisation of the
rows between the two products.

Parity unpinned: the pages give no numbers for these operators.
"""

from __future__ import annotations

import math

import numpy as np

from . import formats as F
from . import quant as Q

TOL = 2.0 ** -18
# An epilogue's own arithmetic: an fp32 power, sum, reciprocal and two
# products, and a power's exponent |v| log2(e) rounded twice.
EPS = 2.0 ** -24
SLOPE = 1.13     # of the activations, at most (gelu's is 1.129)


def route(logits, top_k, bias=None, scoring="softmax", groups=1, top_groups=1, group_top=2, renormalize=True,
          scale=1.0):
    """logits fp64 [T, E] -> (weights fp64 [T, top_k], ids int [T, top_k]), one token at a time."""
    T, E = logits.shape
    weights, ids = np.zeros((T, top_k)), np.full((T, top_k), -1, np.int64)
    big = float(np.finfo(np.float32).max)
    for t in range(T):
        x = np.minimum(logits[t], big)
        b = np.zeros(E) if bias is None else bias
        there = [e for e in range(E) if x[e] > -math.inf and b[e] > -math.inf]
        if not there:
            continue
        s = {}
        if scoring == "softmax":
            top = max(x[e] for e in there)
            total = math.fsum(math.exp(x[e] - top) for e in there)
            s = {e: math.exp(x[e] - top) / total for e in there}
        else:
            s = {e: 1 / (1 + math.exp(-x[e])) if x[e] > -700 else math.exp(x[e]) for e in there}
        c = {e: s[e] + b[e] for e in there}
        if 1 < groups and top_groups < groups:
            size = E // groups
            score = {}
            for g in range(groups):
                inside = sorted((c[e] for e in there if e // size == g), reverse=True)[:group_top]
                if inside:
                    score[g] = sum(inside)
            stay = set(sorted(score, key=lambda g: (-score[g], g))[:top_groups])
            there = [e for e in there if e // size in stay]
        order = sorted(there, key=lambda e: (-c[e], -x[e], e))[:top_k]
        total = math.fsum(s[e] for e in order)
        for j, e in enumerate(order):
            w = s[e]
            if renormalize:
                # (a common factor taken out where all scores vanish)
                w = w / total if total > 1e-290 else math.exp(x[e] - max(x[i] for i in order)) / math.fsum(
                    math.exp(x[i] - max(x[k] for k in order)) for i in order)
            weights[t, j], ids[t, j] = w * scale, e
    return weights, ids


def activation(v, name):
    v = np.asarray(v, np.float64)
    if name == "silu":
        return v / (1 + np.exp(-np.clip(v, -700, 700)))
    if name == "gelu":
        return 0.5 * v * np.vectorize(math.erfc, otypes=[float])(-v / math.sqrt(2))
    if name == "gelu_tanh":
        return 0.5 * v * (1 + np.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
    if name == "relu":
        return np.maximum(v, 0)
    assert name == "none"
    return v


def _activated(v, err, name):
    """act(v) and how far the kernel's may be, its v being within err."""
    a = activation(v, name)
    if name == "none":
        return a, err
    # act's own rounding: the exponent of its power is off by |2 v (1 + v^2 / 22)| roundings, the rest by a few ulps
    own = EPS * (8 + 4 * np.abs(v) * (1 + v * v / 22)) * np.minimum(np.abs(a) + 1e-30, np.abs(v))
    return a, SLOPE * err + own


def product(a, w, bias, act, gated):
    """act(a w^T + bias), gated if asked: (value, bound before the last rounding); a, w fp64."""
    v = a @ w.T
    err = TOL * (np.abs(a) @ np.abs(w).T)
    if bias is not None:
        v, err = v + bias, err + TOL * np.abs(bias)
    if not gated:
        return _activated(v, err, act)
    n = v.shape[1] // 2
    g, eg = _activated(v[:, :n], err[:, :n], act)
    u, eu = v[:, n:], err[:, n:]
    return g * u, eg * np.abs(u) + eu * np.abs(g) + eg * eu + 2 * EPS * np.abs(g * u)


def dequantised(x_bf16):
    return Q.dequant(*Q.quant_1x32(x_bf16))


def linear_act(x_bf16, qw, sw, bias_bf16=None, act="none", gated=False, residual_bf16=None):
    """(out fp64, bound before the cast)."""
    bias = None if bias_bf16 is None else F.bf16_to_f64(bias_bf16)
    y, err = product(dequantised(x_bf16), Q.dequant(qw, sw), bias, act, gated)
    if residual_bf16 is not None:
        y = y + F.bf16_to_f64(residual_bf16)
        err = err + EPS * np.abs(y)
    return y, err


def _scaled(v, b):
    """Blocks v [..., 32] through E2M1 under the scale bytes b [...]."""
    y = np.ldexp(np.abs(v), 127 - b[..., None].astype(np.int64))
    return np.copysign(np.ldexp(F.E2M1_MAGNITUDES[Q.round_to_e2m1_magnitude(y)],
                                b[..., None].astype(np.int64) - 127), v)


def requantised(v, err):
    """bf16(v) through MXFP4, and how far the result may be when v is only
    known to err: the rounding to bf16, the scale's exponent and the rounding
    to E2M1 are monotone, so the extremes of v bound each of them."""
    lo, hi = (F.bf16_to_f64(F.f64_to_bf16(z)).reshape(v.shape[0], -1, 32) for z in (v - err, v + err))
    mid = F.bf16_to_f64(F.f64_to_bf16(v)).reshape(lo.shape)
    most = np.maximum(np.abs(lo), np.abs(hi))
    least = np.where(np.sign(lo) != np.sign(hi), 0.0, np.minimum(np.abs(lo), np.abs(hi)))
    ref = _scaled(mid, Q.scale_byte(np.abs(mid).max(-1)))
    dev = np.zeros_like(ref)
    for b in (Q.scale_byte(least.max(-1)), Q.scale_byte(most.max(-1))):
        for z in (lo, hi):
            dev = np.maximum(dev, np.abs(_scaled(z, b) - ref))
    return ref.reshape(v.shape), dev.reshape(v.shape)


def moe(x_bf16, ids, weights, up, down, up_bias=None, down_bias=None, act="silu", gated=True, residual_bf16=None,
        half=False):
    """up, down: (qw [E, N, K/2], sw [E, N, K/32]); weights fp64.  (out fp64, bound before the cast).

    half: a looser bound, which the library's fp32 rows do not need: a choice's
    row may be held in fp16 with one exponent per 64 columns before it is
    weighted, its largest magnitude scaled into [2^14, 2^15): fp16 keeps 11
    bits, so a value is half a step off, 2^-11 of itself, down to fp16's
    smallest normal number 2^-14, which is 2^-28 of the largest at
    least; below that half a step is 2^-25, 2^-39 of the largest."""
    x = dequantised(x_bf16)
    T, k = ids.shape
    E = up[0].shape[0]
    H = x.shape[1]
    out = np.zeros((T, H)) if residual_bf16 is None else F.bf16_to_f64(residual_bf16)
    err = np.zeros((T, H))
    size = np.abs(out)
    for e in range(E):
        at = [(t, j) for t in range(T) for j in range(k) if ids[t, j] == e]
        if not at:
            continue
        rows = np.array([t for t, _ in at])
        ub = None if up_bias is None else F.bf16_to_f64(up_bias[e])
        h, dev = requantised(*product(x[rows], Q.dequant(up[0][e], up[1][e]), ub, act, gated))
        w = Q.dequant(down[0][e], down[1][e])
        y = h @ w.T
        bound = TOL * (np.abs(h) @ np.abs(w).T) + (1 + TOL) * (dev @ np.abs(w).T)
        if down_bias is not None:
            d = F.bf16_to_f64(down_bias[e])
            y, bound = y + d, bound + TOL * np.abs(d)
        if half:
            bound = bound + 2.0 ** -11 * (np.abs(y) + bound) + 2.0 ** -39 * np.abs(y).max(1, keepdims=True)
        for n, (t, j) in enumerate(at):
            out[t] += weights[t, j] * y[n]
            err[t] += abs(weights[t, j]) * bound[n]
            size[t] += np.abs(weights[t, j] * y[n])
    # a product and a sum per choice, in fp32, and the weight's product with the row's exponent
    return out, err + (2 * k + 1) * EPS * size
