"""GPU parity of the latent-attention operators on arguments whose strides
differ from a packed tensor's: bit for bit what the packed arguments give."""

import numpy as np
import pytest
import torch

import mxfp4_block_scaled_quant_amd as mx
from oracle import attention as A
from tests.helpers import host_bf16_bits, need_gpu
from tests.test_gpu_mla import check, ints, paged, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


def same(got, want):
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("rows", [0, 16, 32, 128])
@pytest.mark.parametrize("B,H", [(3, 16), (70, 5), (4, 40)])
def test_requests_that_share_one_table_row(B, H, rows):
    from mxfp4_block_scaled_quant_amd import ops  # noqa: F401
    cache, table = paged(B + H, [333, 100], 16)
    one, prefix = ints(table[:1]), ints(table[1])
    lens = [333 - (29 * b) % 300 for b in range(B)]
    n, q = ints(lens), randn(B, B, 1, H, 576)
    wide = one.expand(B, -1)
    packed = wide.contiguous()
    assert wide.stride(0) == 0
    try:
        mx.set_mla_rows(rows)
        got = mx.mla_decode(q, cache, wide, n, 0.0625, return_lse=True)
        same(got, mx.mla_decode(q, cache, packed, n, 0.0625, return_lse=True))
        same(torch.ops.mxfp4.mla_decode(q, cache, wide, n, 0.0625), got)
        under = mx.mla_decode_shared_prefix(q, cache, prefix, 100, wide, n, 0.0625, return_lse=True)
        same(under, mx.mla_decode_shared_prefix(q, cache, prefix, 100, packed, n, 0.0625, return_lse=True))
        same(torch.ops.mxfp4.mla_decode_shared_prefix(q, cache, prefix, 100, wide, n, 0.0625), under)
    finally:
        mx.set_mla_rows(0)
    some = [0, B // 2, B - 1]
    check(got[0][some], got[1][some], A.decode(host_bf16_bits(q[some]), host_bf16_bits(cache),
                                               np.repeat(table[:1], 3, 0), [lens[b] for b in some], 0.0625))


def odd(x, *dims):
    """x with a stride of 3 in `dims`, dimensions of one element."""
    strides = list(x.stride())
    for d in dims:
        assert x.shape[d] == 1
        strides[d] = 3
    return x.as_strided(x.shape, strides, x.storage_offset())


def test_strides_of_single_elements_mean_nothing():
    cache, table = paged(2, [300], 16)
    t, n, q = ints(table), ints([300]), randn(1, 1, 1, 16, 576)
    want = mx.mla_decode(q, cache, t, n, 0.0625, return_lse=True)
    out = odd(torch.zeros_like(want[0]), 0, 1)
    same(mx.mla_decode(odd(q, 0, 1), cache, odd(t, 0), n, 0.0625, return_lse=True, out=out), want)
    flat = cache.reshape(-1, 1, 576)                          # pages of one row
    rows = ints((table[:, :, None] * 16 + np.arange(16)).reshape(1, -1))
    same(mx.mla_decode(q, odd(flat, 1), rows, n, 0.0625, return_lse=True), want)
    one = cache[:1].contiguous()                              # one page
    want = mx.mla_decode(q[:, :, :1], one, ints([[0]]), ints([9]), 0.0625, return_lse=True)
    same(mx.mla_decode(odd(q[:, :, :1], 0, 1, 2), odd(one, 0), ints([[0]]), ints([9]), 0.0625, return_lse=True), want)

    cs = randn(3, 10, 64).float()
    kv, w, qr = randn(4, 1, 576), randn(5, 512), randn(6, 1, 16, 64)
    slot, pos = torch.tensor([7], device="cuda"), torch.tensor([3], device="cuda")
    a, b = cache.clone(), cache.clone()
    want = mx.mla_cache_append(kv, w, a, slot, pos, cs, q_pe=qr)
    got = mx.mla_cache_append(odd(kv, 0), w, b, slot, pos, cs, q_pe=odd(qr, 0), q_out=odd(torch.zeros_like(qr), 0))
    assert torch.equal(a, b) and torch.equal(got, want)

    for dn, dv in ((128, 128), (192, 256)):
        q, kn, kp, v = randn(1, 1, 2, dn + 64), randn(2, 1, 2, dn), randn(3, 1, 64), randn(4, 1, 2, dv)
        cu = ints([0, 1])
        for rows in (32, 128):
            try:
                mx.set_mla_prefill_rows(rows)
                want = mx.mla_prefill(q, kn, kp, v, cu, cu, 0.1, return_lse=True)
                got = mx.mla_prefill(odd(q, 0), odd(kn, 0), odd(kp, 0), odd(v, 0), cu, cu, 0.1, return_lse=True,
                                     out=odd(torch.zeros_like(want[0]), 0))
                same(got, want)
                want = mx.mla_prefill(q[:, :1], kn[:, :1], kp, v[:, :1], cu, cu, 0.1, return_lse=True)
                got = mx.mla_prefill(odd(q[:, :1], 0, 1), odd(kn[:, :1], 0, 1), odd(kp, 0), odd(v[:, :1], 0, 1), cu, cu,
                                     0.1, return_lse=True)
                same(got, want)
            finally:
                mx.set_mla_prefill_rows(0)
