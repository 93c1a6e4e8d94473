"""The latent-attention custom ops' fake implementations (no GPU)."""

import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from mxfp4_block_scaled_quant_amd import ops  # noqa: F401  (registers torch.ops.mxfp4)


def t(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="cuda")


def test_decode_and_prefix_shapes():
    with FakeTensorMode():
        table, n, cache = t(3, 9, dtype=torch.int32), t(3, dtype=torch.int32), t(20, 16, 576)
        for q in (t(3, 2, 16, 576), t(3, 16, 576)):
            for out, lse in (torch.ops.mxfp4.mla_decode(q, cache, table, n, 0.1),
                             torch.ops.mxfp4.mla_decode_shared_prefix(q, cache, t(4, dtype=torch.int32), 50, table, n,
                                                                      0.1)):
                assert out.shape == (*q.shape[:-1], 512) and out.dtype == torch.bfloat16
                assert lse.shape == q.shape[:-1] and lse.dtype == torch.float32


def test_prefill_shapes():
    with FakeTensorMode():
        cu = t(3, dtype=torch.int32)
        for dn, dv in ((128, 128), (192, 256)):
            out, lse = torch.ops.mxfp4.mla_prefill(t(7, 4, dn + 64), t(9, 4, dn), t(9, 64), t(9, 4, dv), cu, cu, 0.1)
            assert out.shape == (7, 4, dv) and out.dtype == torch.bfloat16
            assert lse.shape == (7, 4) and lse.dtype == torch.float32


def test_append_returns_nothing():
    with FakeTensorMode():
        i = t(5, dtype=torch.int64)
        assert torch.ops.mxfp4.mla_cache_append(t(5, 576), t(512), t(4, 16, 576), i, i,
                                                t(99, 64, dtype=torch.float32), t(5, 16, 64), t(5, 16, 64)) is None
