"""The rows that wait for their weighted sum are held in fp32 in every form of the experts' products."""

import numpy as np
import pytest

import mxfp4_block_scaled_quant_amd as mx
from oracle import feedforward as D
from oracle import formats as F
from tests.helpers import host_bf16_bits, need_gpu
from tests.test_gpu_moe import device, problem

pytestmark = pytest.mark.gpu


# one launch's sum, streamed rows, tiles; a width of half a wave's columns, several tiles of rows
@pytest.mark.parametrize("T,k,E,H,I", [(3, 2, 4, 256, 64), (40, 4, 16, 256, 64), (96, 4, 16, 256, 64),
                                       (130, 2, 3, 1056, 160), (60, 8, 8, 288, 96), (700, 2, 4, 96, 64)])
@pytest.mark.parametrize("bias", [False, True])
def test_a_residual_that_cancels_the_sum(T, k, E, H, I, bias):
    """Minus the sum, rounded to bf16, as the residual: what is left is under 2^-8 of the sum, and so is the last
    rounding's share of the bound (2^-16 of the sum), so that a row of 11 bits, 2^-12 of it off, would be seen."""
    need_gpu()
    p = problem(T, k, E, H, I, seed=31, bias=bias)
    args = (p["x"], p["ids"], p["weights"].astype(np.float64), p["up"], p["down"], p["up_bias"], p["down_bias"])
    total, _ = D.moe(*args)
    p["residual"] = F.f64_to_bf16(-total)
    ref, err = D.moe(*args, residual_bf16=p["residual"])
    got = F.bf16_to_f64(host_bf16_bits(mx.mxfp4_moe(**device(p))))
    bound = err + 2.0 ** -8 * (np.abs(ref) + err) + 1e-38
    worst = np.max(np.abs(got - ref) / bound)
    assert worst <= 1.0, worst
