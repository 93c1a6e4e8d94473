"""Latent attention at many keys, held to what its roundings add up to.

A probability is rounded to bf16 by at most 2^-8 of itself, and the output is
divided by the sum of the rounded ones, so with errors d_i
    out' - out = sum p_i d_i (v_i - out) / (1 + sum p_i d_i).
The worst case, 2^-8 sum p |v|, has all d_i agree; over many keys they are
independent and even within half a step, so the error's deviation is at most
    s = 2^-8 / sqrt(3) sqrt(sum p_i^2 (v_i - out)^2)
and 7 s, times 1.01 for the denominator, holds for all of some 10^7 outputs
but for odds of 10^-4.  Scores (2^-18 of sum |q k|, which moves a probability
by twice that at most) and the remaining fp32 steps (2^-16) count in full, and
the output is rounded to bf16 once.
"""

import math

import pytest
import torch

import mxfp4_block_scaled_quant_amd as mx
from tests.helpers import need_gpu
from tests.test_gpu_mla import ints, paged, randn

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -8


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


def check(got, lse, q, keys, values, scale, hide=None):
    """Rows of q [R, d] over keys [n, d], values [n, w]; hide [R, n] or None."""
    q, k, v = q.double(), keys.double(), values.double()
    kt = k.t().contiguous()
    z = torch.mm(q, kt) * scale
    size = torch.mm(q.abs(), kt.abs()) * scale
    if hide is not None:
        z = z.masked_fill(hide, -math.inf)
        size = size.masked_fill(hide, 0)
    ref_lse = torch.logsumexp(z, 1)
    p = torch.exp(z - ref_lse[:, None])
    out = torch.mm(p, v)
    square = p * p
    spread = torch.mm(square, v * v) - 2 * out * torch.mm(square, v) + out * out * square.sum(1, keepdim=True)
    ez = 2.0 ** -18 * size.amax(1, keepdim=True)
    tol = 7 * 1.01 * HALF / math.sqrt(3) * spread.clamp(min=0).sqrt() + (2.0 ** -16 + 2 * ez) * torch.mm(p, v.abs())
    tol = tol + HALF * (out.abs() + tol)
    off = (got.double() - out).abs()
    assert torch.isfinite(got).all() and (off <= tol).all(), f"off by {(off / tol).max().item():.3g} of its tolerance"
    off = (lse.double() - ref_lse).abs()
    assert (off <= ez[:, 0] + 2.0 ** -20 * (1 + ref_lse.abs())).all(), f"lse off by {off.max().item():.3g}"


@pytest.mark.parametrize("B,S,H,n,page", [(1, 1, 16, 40001, 64), (3, 1, 16, 9000, 16), (2, 1, 32, 20011, 64),
                                          (2, 1, 64, 5003, 1), (1, 1, 128, 12345, 64), (4, 3, 128, 6000, 64)])
def test_decode(B, S, H, n, page):
    lens = [n - 13 * i for i in range(B)]
    cache, table = paged(n, lens, page)
    q = randn(H + 1, B, S, H, 576)
    t = ints(table)
    out, lse = mx.mla_decode(q, cache, t, ints(lens), 0.05, return_lse=True)
    for b in range(B):
        rows = cache[t[b].long()].reshape(-1, 576)[:lens[b]]
        for s in range(S):
            k = rows[:lens[b] - S + 1 + s]
            check(out[b, s], lse[b, s], q[b, s], k, k[:, :512], 0.05)


def under_prefix(B, S, H, prefix, lens, some):
    cache, table = paged(prefix, lens + [prefix], 64)
    ptab, t, n = ints(table[-1]), ints(table[:-1]), ints(lens)
    q = randn(H + 2, B, S, H, 576)
    out, lse = mx.mla_decode_shared_prefix(q, cache, ptab, prefix, t, n, 0.05, return_lse=True)
    again = mx.mla_decode_shared_prefix(q, cache, ptab, prefix, t, n, 0.05, return_lse=True)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    shared = cache[ptab.long()].reshape(-1, 576)[:prefix]
    for b in some:
        rows = torch.cat([shared, cache[t[b].long()].reshape(-1, 576)[:lens[b]]])
        for s in range(S):
            k = rows[:prefix + max(0, lens[b] - S + 1 + s)]
            check(out[b, s], lse[b, s], q[b, s], k, k[:, :512], 0.05)


def test_long_prefix():
    under_prefix(24, 1, 16, 12001, [1 + 37 * i for i in range(24)], (0, 11, 23))


@pytest.mark.parametrize("rows,prefix", [(0, 100), (0, 301), (16, 301), (32, 301), (128, 2000)])
def test_more_prefix_rows_than_workgroups_hold_at_once(rows, prefix):
    # 65 requests of 4 tokens x 128 heads, 33280 query rows: the prefix has
    # more row blocks than there are workgroups (260 of 128 rows)
    lens = [(91 * i) % 230 for i in range(65)]
    lens[3] = 0
    try:
        mx.set_mla_rows(rows)
        under_prefix(65, 4, 128, prefix, lens, (0, 3, 31, 64))
    finally:
        mx.set_mla_rows(0)


@pytest.mark.parametrize("rows", [32, 128])
@pytest.mark.parametrize("n,keys,H,dn,dv,causal", [(1000, 1000, 3, 128, 128, True), (777, 2277, 2, 192, 256, True),
                                                   (513, 3513, 8, 128, 128, True), (300, 5000, 3, 128, 128, False),
                                                   (257, 3001, 2, 192, 256, False)])
def test_prefill(n, keys, H, dn, dv, causal, rows):
    q, kn, kp, v = randn(1, n, H, dn + 64), randn(2, keys, H, dn), randn(3, keys, 64), randn(4, keys, H, dv)
    try:
        mx.set_mla_prefill_rows(rows)
        out, lse = mx.mla_prefill(q, kn, kp, v, ints([0, n]), ints([0, keys]), 0.08, causal=causal, return_lse=True)
    finally:
        mx.set_mla_prefill_rows(0)
    hide = torch.ones((n, keys), device="cuda").triu(keys - n + 1).bool() if causal else None
    for h in range(H):
        check(out[:, h], lse[:, h], q[:, h], torch.cat([kn[:, h], kp], 1), v[:, h], 0.08, hide)
