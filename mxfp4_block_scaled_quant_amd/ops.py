"""torch custom operators over the C ABI, with fake (meta) implementations.

The registered quantisation and GEMM ops of P2 §2 let the serving framework
trace, compile and capture the FP4 linear; these are their counterparts for
this library.  Each op's real implementation is the ctypes binding (every
step runs in the HIP kernels); its fake implementation only states output
shapes and dtypes, computed from the same layout rules as the library's size
queries, and works with symbolic sizes.

    torch.ops.mxfp4.quant_1x32(x, layout) -> (q, scales)
    torch.ops.mxfp4.preshuffle_weight(w_fp4, w_scales, N, K, batch) -> (w_pre, ws_pre)
    torch.ops.mxfp4.gemm_a4w4(a, a_scales, w_pre, ws_pre, M, N, K, bias, out_dtype) -> [M, N]
    torch.ops.mxfp4.linear(x, w_pre, ws_pre, N, bias, out_dtype) -> [M, N]
    torch.ops.mxfp4.gemm_a4w4_mxfp4_out(a, a_scales, w_pre, ws_pre, M, N, K, bias)
        -> (q [M, N/2], scales [M, N/32])
    torch.ops.mxfp4.shuffle_scales(scales, rows, K) -> GEMM-layout scales
    torch.ops.mxfp4.linear_prequantized(x_fp4, x_scales, w_pre, ws_pre, N, bias,
        out_dtype) -> [M, N]
    torch.ops.mxfp4.a16wfp4_bmm(x, w_pre, ws_pre, N, batch_major, out_dtype)
        -> [B, M, N] or [M, B, N]
    torch.ops.mxfp4.mla_cache_append(kv, norm_weight, cache, slots, positions,
        cos_sin, q_pe, q_out, eps, interleaved) -> None   (writes cache and q_out)
    torch.ops.mxfp4.mla_decode(q, cache, block_table, lengths, scale)
        -> (out [B, S, H, 512], lse [B, S, H])
    torch.ops.mxfp4.mla_decode_shared_prefix(q, cache, prefix_table, prefix_len,
        block_table, lengths, scale) -> (out, lse)
    torch.ops.mxfp4.mla_prefill(q, k_nope, k_pe, v, cu_q, cu_k, scale, causal)
        -> (out [Tq, H, dv], lse [Tq, H])
    torch.ops.mxfp4.moe_route(logits, top_k, bias, scoring, groups, top_groups, group_top,
        renormalize, scale) -> (weights [T, top_k], ids [T, top_k])
    torch.ops.mxfp4.moe(x, ids, weights, up_w, up_ws, down_w, down_ws, experts, inner,
        up_bias, down_bias, activation, gated, residual) -> [T, hidden]
    torch.ops.mxfp4.linear_act(x, w_pre, ws_pre, N, bias, activation, gated, residual,
        out_dtype) -> [M, N] ([M, N/2] gated)

mla_cache_append writes the cache and q_out it is given; no other op mutates
its inputs, and none has an autograd formula (the path is inference only).
"""

from __future__ import annotations

from typing import Optional, Tuple

import torch
from torch import Tensor

from . import (MXFP4_LAYOUT_GEMM, MXFP4_LAYOUT_ROWMAJOR, a16wfp4_bmm, mxfp4_gemm_a4w4,
               MXFP4Weight, mla_cache_append, mla_decode, mla_decode_shared_prefix, mla_prefill, moe_route,
               mxfp4_gemm_a4w4_mxfp4_out, mxfp4_linear, mxfp4_linear_act, mxfp4_linear_prequantized, mxfp4_moe,
               mxfp4_preshuffle_weight, mxfp4_quant_1x32, mxfp4_shuffle_scales)

__all__ = ["gemm_data_bytes", "gemm_scale_bytes"]


def _cdiv(a, b):
    return (a + b - 1) // b


def gemm_data_bytes(rows, K):
    """Bytes of packed FP4 in the GEMM data layout: whole 1 KiB units of
    16 rows x 128 K (rows and K padded)."""
    return _cdiv(rows, 16) * _cdiv(K, 128) * 1024


def gemm_scale_bytes(rows, K):
    """Bytes of E8M0 scales in the GEMM scale layout: 256-byte units of
    16 rows x 4 K-steps."""
    return _cdiv(rows, 16) * _cdiv(_cdiv(K, 128), 4) * 256


@torch.library.custom_op("mxfp4::quant_1x32", mutates_args=())
def quant_1x32(x: Tensor, layout: int) -> Tuple[Tensor, Tensor]:
    q, s = mxfp4_quant_1x32(x, layout)
    return q, s


@quant_1x32.register_fake
def _(x, layout):
    M, K = x.shape
    if layout == MXFP4_LAYOUT_ROWMAJOR:
        return (x.new_empty((M, K // 2), dtype=torch.uint8),
                x.new_empty((M * (K // 32),), dtype=torch.uint8))
    if layout == MXFP4_LAYOUT_GEMM:
        return (x.new_empty((gemm_data_bytes(M, K),), dtype=torch.uint8),
                x.new_empty((gemm_scale_bytes(M, K),), dtype=torch.uint8))
    raise ValueError(f"unknown layout {layout}")


@torch.library.custom_op("mxfp4::preshuffle_weight", mutates_args=())
def preshuffle_weight(w_fp4: Tensor, w_scales: Tensor, N: int, K: int,
                      batch: int = 1) -> Tuple[Tensor, Tensor]:
    w_pre, ws_pre = mxfp4_preshuffle_weight(w_fp4, w_scales, N, K, batch=batch)
    return w_pre, ws_pre


@preshuffle_weight.register_fake
def _(w_fp4, w_scales, N, K, batch=1):
    return (w_fp4.new_empty((batch * gemm_data_bytes(N, K),), dtype=torch.uint8),
            w_fp4.new_empty((batch * gemm_scale_bytes(N, K),), dtype=torch.uint8))


@torch.library.custom_op("mxfp4::gemm_a4w4", mutates_args=())
def gemm_a4w4(a: Tensor, a_scales: Tensor, w_pre: Tensor, ws_pre: Tensor, M: int, N: int,
              K: int, bias: Optional[Tensor] = None,
              out_dtype: torch.dtype = torch.bfloat16) -> Tensor:
    return mxfp4_gemm_a4w4(a, a_scales, w_pre, ws_pre, M, N, K, bias, out_dtype)


@gemm_a4w4.register_fake
def _(a, a_scales, w_pre, ws_pre, M, N, K, bias=None, out_dtype=torch.bfloat16):
    return a.new_empty((M, N), dtype=out_dtype)


@torch.library.custom_op("mxfp4::linear", mutates_args=())
def linear(x: Tensor, w_pre: Tensor, ws_pre: Tensor, N: int, bias: Optional[Tensor] = None,
           out_dtype: torch.dtype = torch.bfloat16) -> Tensor:
    return mxfp4_linear(x, w_pre, ws_pre, N, bias, out_dtype)


@linear.register_fake
def _(x, w_pre, ws_pre, N, bias=None, out_dtype=torch.bfloat16):
    return x.new_empty((x.shape[0], N), dtype=out_dtype)


@torch.library.custom_op("mxfp4::gemm_a4w4_mxfp4_out", mutates_args=())
def gemm_a4w4_mxfp4_out(a: Tensor, a_scales: Tensor, w_pre: Tensor, ws_pre: Tensor, M: int,
                        N: int, K: int, bias: Optional[Tensor] = None) -> Tuple[Tensor, Tensor]:
    q, s = mxfp4_gemm_a4w4_mxfp4_out(a, a_scales, w_pre, ws_pre, M, N, K, bias)
    return q, s


@gemm_a4w4_mxfp4_out.register_fake
def _(a, a_scales, w_pre, ws_pre, M, N, K, bias=None):
    return (a.new_empty((M, N // 2), dtype=torch.uint8), a.new_empty((M, N // 32), dtype=torch.uint8))


@torch.library.custom_op("mxfp4::shuffle_scales", mutates_args=())
def shuffle_scales(scales: Tensor, rows: int, K: int) -> Tensor:
    return mxfp4_shuffle_scales(scales, rows, K)


@shuffle_scales.register_fake
def _(scales, rows, K):
    return scales.new_empty((gemm_scale_bytes(rows, K),), dtype=torch.uint8)


@torch.library.custom_op("mxfp4::linear_prequantized", mutates_args=())
def linear_prequantized(x_fp4: Tensor, x_scales: Tensor, w_pre: Tensor, ws_pre: Tensor, N: int,
                        bias: Optional[Tensor] = None,
                        out_dtype: torch.dtype = torch.bfloat16) -> Tensor:
    return mxfp4_linear_prequantized(x_fp4, x_scales, w_pre, ws_pre, N, bias, out_dtype)


@linear_prequantized.register_fake
def _(x_fp4, x_scales, w_pre, ws_pre, N, bias=None, out_dtype=torch.bfloat16):
    return x_fp4.new_empty((x_fp4.shape[0], N), dtype=out_dtype)


@torch.library.custom_op("mxfp4::a16wfp4_bmm", mutates_args=())
def bmm(x: Tensor, w_pre: Tensor, ws_pre: Tensor, N: int, batch_major: bool = False,
        out_dtype: torch.dtype = torch.bfloat16) -> Tensor:
    return a16wfp4_bmm(x, w_pre, ws_pre, N, batch_major=batch_major, out_dtype=out_dtype)


@bmm.register_fake
def _(x, w_pre, ws_pre, N, batch_major=False, out_dtype=torch.bfloat16):
    B, M, _ = x.shape
    shape = (M, B, N) if batch_major else (B, M, N)
    return x.new_empty(shape, dtype=out_dtype)


@torch.library.custom_op("mxfp4::mla_cache_append", mutates_args=("cache", "q_out"))
def cache_append(kv: Tensor, norm_weight: Tensor, cache: Tensor, slots: Tensor, positions: Tensor, cos_sin: Tensor,
                 q_pe: Optional[Tensor] = None, q_out: Optional[Tensor] = None, eps: float = 1e-6,
                 interleaved: bool = True) -> None:
    if (q_pe is None) != (q_out is None):
        raise ValueError("q_pe and q_out are given together")
    mla_cache_append(kv, norm_weight, cache, slots, positions, cos_sin, q_pe, q_out, eps, interleaved)


@cache_append.register_fake
def _(kv, norm_weight, cache, slots, positions, cos_sin, q_pe=None, q_out=None, eps=1e-6, interleaved=True):
    return None


@torch.library.custom_op("mxfp4::mla_decode", mutates_args=())
def decode(q: Tensor, cache: Tensor, block_table: Tensor, lengths: Tensor, scale: float) -> Tuple[Tensor, Tensor]:
    out, lse = mla_decode(q, cache, block_table, lengths, scale, return_lse=True)
    return out, lse


def _decode_fake(q):
    return (q.new_empty((*q.shape[:-1], 512), dtype=torch.bfloat16),
            q.new_empty(tuple(q.shape[:-1]), dtype=torch.float32))


@decode.register_fake
def _(q, cache, block_table, lengths, scale):
    return _decode_fake(q)


@torch.library.custom_op("mxfp4::mla_decode_shared_prefix", mutates_args=())
def decode_shared_prefix(q: Tensor, cache: Tensor, prefix_table: Tensor, prefix_len: int, block_table: Tensor,
                         lengths: Tensor, scale: float) -> Tuple[Tensor, Tensor]:
    out, lse = mla_decode_shared_prefix(q, cache, prefix_table, prefix_len, block_table, lengths, scale,
                                        return_lse=True)
    return out, lse


@decode_shared_prefix.register_fake
def _(q, cache, prefix_table, prefix_len, block_table, lengths, scale):
    return _decode_fake(q)


@torch.library.custom_op("mxfp4::mla_prefill", mutates_args=())
def prefill(q: Tensor, k_nope: Tensor, k_pe: Tensor, v: Tensor, cu_q: Tensor, cu_k: Tensor, scale: float,
            causal: bool = True) -> Tuple[Tensor, Tensor]:
    out, lse = mla_prefill(q, k_nope, k_pe, v, cu_q, cu_k, scale, causal=causal, return_lse=True)
    return out, lse


@prefill.register_fake
def _(q, k_nope, k_pe, v, cu_q, cu_k, scale, causal=True):
    T, H = q.shape[:2]
    return (q.new_empty((T, H, v.shape[2]), dtype=torch.bfloat16), q.new_empty((T, H), dtype=torch.float32))


@torch.library.custom_op("mxfp4::moe_route", mutates_args=())
def route(logits: Tensor, top_k: int, bias: Optional[Tensor] = None, scoring: str = "softmax", groups: int = 1,
          top_groups: int = 1, group_top: int = 2, renormalize: bool = True,
          scale: float = 1.0) -> Tuple[Tensor, Tensor]:
    return moe_route(logits, top_k, bias, scoring, groups, top_groups, group_top, renormalize, scale)


@route.register_fake
def _(logits, top_k, bias=None, scoring="softmax", groups=1, top_groups=1, group_top=2, renormalize=True, scale=1.0):
    T = logits.shape[0]
    return logits.new_empty((T, top_k), dtype=torch.float32), logits.new_empty((T, top_k), dtype=torch.int32)


@torch.library.custom_op("mxfp4::moe", mutates_args=())
def moe(x: Tensor, ids: Tensor, weights: Tensor, up_w: Tensor, up_ws: Tensor, down_w: Tensor, down_ws: Tensor,
        experts: int, inner: int, up_bias: Optional[Tensor] = None, down_bias: Optional[Tensor] = None,
        activation: str = "silu", gated: bool = True, residual: Optional[Tensor] = None) -> Tensor:
    hidden = x.shape[1]
    up = MXFP4Weight(up_w, up_ws, 2 * inner if gated else inner, hidden, experts)
    return mxfp4_moe(x, ids, weights, up, MXFP4Weight(down_w, down_ws, hidden, inner, experts), up_bias, down_bias,
                     activation, gated, residual)


@moe.register_fake
def _(x, ids, weights, up_w, up_ws, down_w, down_ws, experts, inner, up_bias=None, down_bias=None, activation="silu",
      gated=True, residual=None):
    return x.new_empty((x.shape[0], x.shape[1]))


@torch.library.custom_op("mxfp4::linear_act", mutates_args=())
def linear_act(x: Tensor, w_pre: Tensor, ws_pre: Tensor, N: int, bias: Optional[Tensor] = None,
               activation: str = "none", gated: bool = False, residual: Optional[Tensor] = None,
               out_dtype: torch.dtype = torch.bfloat16) -> Tensor:
    return mxfp4_linear_act(x, w_pre, ws_pre, N, bias, activation, gated, residual, out_dtype)


@linear_act.register_fake
def _(x, w_pre, ws_pre, N, bias=None, activation="none", gated=False, residual=None, out_dtype=torch.bfloat16):
    return x.new_empty((x.shape[0], N // 2 if gated else N), dtype=out_dtype)
