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


def test_appended_rows():
    """A wave per token: all but the last few tokens' rows are padding."""
    _room(110)
    T, n = 2 ** 26 + 64, 96
    g = torch.Generator(device="cuda").manual_seed(3)
    kv = torch.empty((T, 576), dtype=torch.bfloat16, device="cuda")
    kv[-n:] = torch.randn((n, 576), generator=g, device="cuda").bfloat16()
    q = torch.empty((T, 1, 64), dtype=torch.bfloat16, device="cuda")
    q[-n:] = torch.randn((n, 1, 64), generator=g, device="cuda").bfloat16()
    slots = torch.full((T,), -1, dtype=torch.int64, device="cuda")
    slots[-n:] = torch.arange(n, device="cuda")
    positions = torch.full((T,), 1 << 20, dtype=torch.int64, device="cuda")     # outside the table: nothing is written
    positions[-n:] = torch.arange(n, device="cuda")
    angles = torch.randn((n, 64), generator=g, device="cuda")
    norm = torch.ones(512, dtype=torch.bfloat16, device="cuda")
    cache, want = (torch.zeros((2, 64, 576), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    want_q = mx.mla_cache_append(kv[-n:], norm, want, slots[-n:], positions[-n:], angles, q[-n:])
    got_q = mx.mla_cache_append(kv, norm, cache, slots, positions, angles, q)
    assert torch.equal(cache, want) and torch.equal(got_q[-n:], want_q)
    assert want.any()


def test_a_batched_product_of_too_many_columns_is_refused():
    _room(70)
    B, M, N, K = 16, 64, 2 ** 24 + 4096, 32
    w = torch.empty((mx.weight_bytes(B, N, K),), dtype=torch.uint8, device="cuda")
    s = torch.empty((mx.weight_scale_bytes(B, N, K),), dtype=torch.uint8, device="cuda")
    x = torch.zeros((B, M, K), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(Exception, match="a16wfp4_bmm"):
        mx.a16wfp4_bmm(x, w, s, N)
