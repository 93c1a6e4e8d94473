"""Refusals of calls that one launch cannot do, on the CPU."""

import ctypes

import mxfp4_block_scaled_quant_amd as mx

P = ctypes.c_void_p(0x10000)
SHAPE = 2


def test_prefill_blocks_past_32_bits():
    def call(B, H, Tq):
        return mx.lib().mla_prefill(P, H * 192, 192, P, H * 128, 128, P, 64, P, H * 128, 128, P, P, B, H, Tq, Tq, 128, 128,
                                    1, 0.1, P, H * 128, 128, None, None)

    assert call(2 ** 17, 128, 2 ** 17) == SHAPE and call(2 ** 24, 1, 2 ** 24) == SHAPE
    assert call(1, 128, 2 ** 24) == SHAPE
    assert call(2 ** 16, 128, 2 ** 16) != SHAPE and call(1, 128, 2 ** 23) != SHAPE
