"""Calls whose threads are more than the 2^32 work items that one launch does: every output is written."""

import pytest
import torch

import mxfp4_block_scaled_quant_amd as mx
from tests.helpers import need_gpu

pytestmark = pytest.mark.gpu


def _room(gib):
    need_gpu()
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gib * 2 ** 30:
        pytest.skip(f"needs {gib} GiB")


def test_quantised_rows():
    """A flat tensor as rows of one block: 2^28 rows, a wave of four rows."""
    _room(40)
    M, K = 2 ** 28 + 4096, 32
    base = torch.randn(4096, K, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").bfloat16()
    q, s = mx.mxfp4_quant_1x32(base.repeat(M // 4096, 1), mx.MXFP4_LAYOUT_ROWMAJOR)
    rq, rs = mx.mxfp4_quant_1x32(base, mx.MXFP4_LAYOUT_ROWMAJOR)
    assert (q.view(-1, 4096, K // 2) == rq).all() and (s.view(-1, rs.numel()) == rs.view(-1)).all()


def test_preshuffled_stacks():
    """A stack of weights: a thread per 16 bytes of data and per four scales."""
    _room(70)
    batch, N, K = 2 ** 16 + 5, 8192, 32
    g = torch.Generator(device="cuda").manual_seed(2)
    w = torch.randint(0, 256, (1, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = torch.randint(100, 140, (1, N, K // 32), generator=g, device="cuda", dtype=torch.uint8)
    rw, rs = mx.mxfp4_preshuffle_weight(w, s, N, K)
    pw, ps = mx.mxfp4_preshuffle_weight(w.repeat(batch, 1, 1), s.repeat(batch, 1, 1), N, K, batch=batch)
    for got, ref in ((pw, rw), (ps, rs)):
        for part in got.view(batch, -1).split(4096):
            assert (part == ref.view(-1)).all()
