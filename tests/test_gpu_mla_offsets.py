"""Offsets of mla_prefill's packed sequences that lie outside the tensors: no
row outside the output is written, and what is written is finite."""

import pytest
import torch

import mxfp4_block_scaled_quant_amd as mx
from tests.helpers import need_gpu
from tests.test_gpu_mla import ints, randn

pytestmark = pytest.mark.gpu

LOW, HIGH = -2 ** 31, 2 ** 31 - 1
OFFSETS = [
    [LOW, HIGH],                  # one sequence of 2^32 - 1 rows: its last block's row number wraps
    [0, HIGH],
    [LOW, 0, HIGH],
    [50, -7, HIGH, LOW, 20],
    [LOW if i % 2 else HIGH for i in range(71)],     # totals of blocks that wrap
    [LOW] + [HIGH] * 3 + [0],
    [9, 9, 9],
]


@pytest.mark.parametrize("rows", [32, 128])
@pytest.mark.parametrize("offsets", OFFSETS)
@pytest.mark.parametrize("causal", [True, False])
def test_wild_offsets_stay_inside_the_tensors(offsets, rows, causal):
    need_gpu()
    T, H, guard = 60, 2, 4096
    for dn, dv in ((128, 128), (192, 256)):
        q, kn, kp, v = randn(1, T, H, dn + 64), randn(2, T, H, dn), randn(3, T, 64), randn(4, T, H, dv)
        room = torch.full((T + 2 * guard, H, dv), 7.0, dtype=torch.bfloat16, device="cuda")
        logs = torch.full((T + 2 * guard, H), 7.0, device="cuda")
        cu, ok = ints(offsets), ints([i * T // (len(offsets) - 1) for i in range(len(offsets))])
        try:
            mx.set_mla_prefill_rows(rows)
            for cu_q, cu_k in ((cu, cu), (cu, ok), (ok, cu)):
                mx.mla_prefill(q, kn, kp, v, cu_q, cu_k, 0.1, causal=causal, out=room[guard:guard + T],
                               lse=logs[guard:guard + T])
                torch.cuda.synchronize()
        finally:
            mx.set_mla_prefill_rows(0)
        for outside in (room[:guard], room[guard + T:], logs[:guard], logs[guard + T:]):
            assert (outside == 7).all()
        assert torch.isfinite(room[guard:guard + T]).all()
