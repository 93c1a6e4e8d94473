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
