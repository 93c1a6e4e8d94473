"""Latent attention from its definition, fp64 (test infrastructure only).

Inputs are bf16 bit patterns (uint16 arrays) or fp64 arrays; every function
also returns what the tolerance of a kernel with bf16 probabilities needs:
``A = sum p |v|``, the weighted magnitude of the values, and ``E``, the
largest ``scale * sum |q_j k_j|`` over a row's visible keys.
"""

from __future__ import annotations

import numpy as np

from . import formats as F


def f64(x):
    return F.bf16_to_f64(x) if x.dtype == np.uint16 else np.asarray(x, np.float64)


def attend_row(q, keys, values, scale):
    """One query over its visible keys: (out, lse, A, E)."""
    if len(keys) == 0:
        return np.zeros(values.shape[1]), -np.inf, np.zeros(values.shape[1]), 0.0
    z = scale * (keys @ q)
    top = z.max()
    w = np.exp(z - top)
    total = w.sum()
    p = w / total
    return p @ values, top + np.log(total), p @ np.abs(values), float(scale * (np.abs(keys) @ np.abs(q)).max())


def paged_rows(cache, table, n):
    """The first n rows behind a page table; rows of pages the cache lacks are left out (None)."""
    pages, size = cache.shape[:2]
    rows = []
    for t in range(n):
        p = int(table[t // size])
        rows.append(cache[p, t % size] if 0 <= p < pages else None)
    return rows


def decode(q, cache, table, lengths, scale, prefix_table=None, prefix_len=0):
    """q [B, S, H, 576], cache [P, page, 576], table [B, W], lengths [B]."""
    q, cache = f64(q), f64(cache)
    B, S, H, D = q.shape
    L = 512
    out, lse = np.zeros((B, S, H, L)), np.zeros((B, S, H))
    A, E = np.zeros((B, S, H, L)), np.zeros((B, S, H))
    shared = paged_rows(cache, prefix_table, prefix_len) if prefix_len else []
    for b in range(B):
        n = min(max(int(lengths[b]), 0), table.shape[1] * cache.shape[1])
        own = paged_rows(cache, table[b], n)
        for s in range(S):
            rows = [r for r in shared + own[:max(0, n - S + 1 + s)] if r is not None]
            keys = np.array(rows) if rows else np.zeros((0, D))
            for h in range(H):
                out[b, s, h], lse[b, s, h], A[b, s, h], E[b, s, h] = attend_row(q[b, s, h], keys, keys[:, :L], scale)
    return out, lse, A, E


def prefill(q, k_nope, k_pe, v, cu_q, cu_k, scale, causal=True):
    q, k_nope, k_pe, v = f64(q), f64(k_nope), f64(k_pe), f64(v)
    T, H, _ = q.shape
    out, lse = np.zeros((T, H, v.shape[2])), np.zeros((T, H))
    A, E = np.zeros_like(out), np.zeros((T, H))
    for b in range(len(cu_q) - 1):
        ks, nk, nq = int(cu_k[b]), int(cu_k[b + 1] - cu_k[b]), int(cu_q[b + 1] - cu_q[b])
        for h in range(H):
            keys = np.concatenate([k_nope[ks:ks + nk, h], k_pe[ks:ks + nk]], 1)
            vals = v[ks:ks + nk, h]
            for i in range(nq):
                t, n = int(cu_q[b]) + i, max(0, nk - nq + 1 + i) if causal else nk
                out[t, h], lse[t, h], A[t, h], E[t, h] = attend_row(q[t, h], keys[:n], vals[:n], scale)
    return out, lse, A, E


def rotate(x, angle_cos, angle_sin, interleaved):
    """Rotate the 32 pairs of the last axis of x [..., 64]."""
    y = np.empty_like(x)
    for i in range(32):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, 32 + i)
        y[..., a] = x[..., a] * angle_cos[..., i] - x[..., b] * angle_sin[..., i]
        y[..., b] = x[..., b] * angle_cos[..., i] + x[..., a] * angle_sin[..., i]
    return y


def cache_rows(kv, weight, cos_sin, positions, eps, interleaved):
    """The rows mla_cache_append writes, before rounding: [T, 576]."""
    kv, weight = f64(kv), f64(weight)
    c = kv[:, :512]
    c = c / np.sqrt((c * c).mean(1, keepdims=True) + eps) * weight
    a = np.asarray(cos_sin, np.float64)[positions]
    return np.concatenate([c, rotate(kv[:, 512:], a[:, :32], a[:, 32:], interleaved)], 1)
