"""Latent attention between the absorbed products: the cache write, attention
over the paged latents (with or without a prefix that all requests share) and
attention over expanded keys and values.

Same rules as the rest of the binding: every tensor is checked on the host,
outputs and the workspace are allocated with torch where they are not given,
and the HIP kernels behind the C ABI (``include/mxfp4.h``) run on the current
stream.  A cache is bf16 ``[pages, page_size, 576]``: the normed latent (512
values) and the rotated key part (64).
"""

from __future__ import annotations

from typing import Optional

import torch

from . import _check, _ptr, _require_cuda, _stream, lib

LATENT_DIM = 512
ROPE_DIM = 64
ROW_DIM = LATENT_DIM + ROPE_DIM


def _require(t: torch.Tensor, name: str, dtype: torch.dtype, shape, device: torch.device) -> None:
    """t has this dtype and shape (-1: any size) on `device` and unit stride along its last dimension."""
    if t.dtype != dtype or t.device != device or t.dim() != len(shape) or any(
            w >= 0 and n != w for n, w in zip(t.shape, shape)):
        want = ", ".join("any" if w < 0 else str(w) for w in shape)
        raise ValueError(f"{name} must be {dtype} [{want}] on {device}, got {t.dtype} {tuple(t.shape)} on {t.device}")
    if t.numel() and t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must have unit stride along its last dimension")


def _require_contiguous(t: torch.Tensor, name: str) -> None:
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def mla_decode_workspace_bytes(B: int, S: int, H: int, max_tokens: int, prefix_len: int = 0) -> int:
    return int(lib().mla_decode_workspace_bytes(B, S, H, max_tokens, prefix_len))


def mla_cache_append(kv: torch.Tensor, norm_weight: torch.Tensor, cache: torch.Tensor, slots: torch.Tensor,
                     positions: torch.Tensor, cos_sin: torch.Tensor, q_pe: Optional[torch.Tensor] = None,
                     q_out: Optional[torch.Tensor] = None, eps: float = 1e-6,
                     interleaved: bool = True) -> Optional[torch.Tensor]:
    """Write T tokens' rows into the cache and rotate their queries; returns ``q_out``.

    kv bf16 [T, 576] (any row stride): the latent, normed here with
    ``norm_weight`` (bf16 [512]), and the key part, rotated by ``positions``
    (int64 [T]) through ``cos_sin`` (fp32 [max_position, 64]: cos of 32
    angles, then their sin).  ``slots`` int64 [T]: page * page_size + row; a
    negative slot writes no row.  ``q_pe`` bf16 [T, H, 64] (any strides) is
    rotated into ``q_out`` (allocated when not given; it may be ``q_pe``
    itself, or the last 64 columns of an absorbed query).
    """
    _require_cuda(kv, "kv")
    dev = kv.device
    _require(kv, "kv", torch.bfloat16, (-1, ROW_DIM), dev)
    T = kv.shape[0]
    _require(norm_weight, "norm_weight", torch.bfloat16, (LATENT_DIM,), dev)
    _require(cache, "cache", torch.bfloat16, (-1, -1, ROW_DIM), dev)
    _require(slots, "slots", torch.int64, (T,), dev)
    _require(positions, "positions", torch.int64, (T,), dev)
    _require(cos_sin, "cos_sin", torch.float32, (-1, ROPE_DIM), dev)
    _require_contiguous(cos_sin, "cos_sin")
    H = 0
    if q_pe is not None:
        _require(q_pe, "q_pe", torch.bfloat16, (T, -1, ROPE_DIM), dev)
        H = q_pe.shape[1]
        if q_out is None:
            q_out = torch.empty((T, H, ROPE_DIM), dtype=torch.bfloat16, device=dev)
        else:
            _require(q_out, "q_out", torch.bfloat16, (T, H, ROPE_DIM), dev)
    elif q_out is not None:
        raise ValueError("q_out is given without q_pe")
    with_q = q_pe is not None and H > 0
    _check("mla_cache_append", lib().mla_cache_append(
        _ptr(kv), kv.stride(0), _ptr(norm_weight), eps, _ptr(cos_sin), cos_sin.shape[0], _ptr(positions),
        _ptr(slots), int(interleaved),
        _ptr(q_pe) if with_q else None, q_pe.stride(0) if with_q else 0, q_pe.stride(1) if with_q else 0,
        _ptr(q_out) if with_q else None, q_out.stride(0) if with_q else 0, q_out.stride(1) if with_q else 0,
        _ptr(cache), cache.shape[0], cache.shape[1], cache.stride(0), cache.stride(1), T, H, _stream(dev)))
    return q_out


def _decode(fn, q, cache, prefix, block_table, lengths, scale, return_lse, out, lse, workspace):
    _require_cuda(q, "q")
    dev = q.device
    three = q.dim() == 3
    if three:
        q = q.unsqueeze(1)
        out = None if out is None else out.unsqueeze(1)
        lse = None if lse is None else lse.unsqueeze(1)
    _require(q, "q", torch.bfloat16, (-1, -1, -1, ROW_DIM), dev)
    B, S, H, _ = q.shape
    _require(cache, "cache", torch.bfloat16, (-1, -1, ROW_DIM), dev)
    _require(block_table, "block_table", torch.int32, (B, -1), dev)
    _require(lengths, "lengths", torch.int32, (B,), dev)
    _require_contiguous(lengths, "lengths")
    pages, page_size = cache.shape[0], cache.shape[1]
    width = block_table.shape[1]
    prefix_table, prefix_len = prefix if prefix else (None, 0)
    if prefix_table is not None:
        _require(prefix_table, "prefix_table", torch.int32, (-1,), dev)
        _require_contiguous(prefix_table, "prefix_table")
        if not 0 <= prefix_len <= prefix_table.shape[0] * page_size:
            raise ValueError(f"prefix_len {prefix_len} does not fit prefix_table's {prefix_table.shape[0]} pages")
    if out is None:
        out = torch.empty((B, S, H, LATENT_DIM), dtype=torch.bfloat16, device=dev)
    else:
        _require(out, "out", torch.bfloat16, (B, S, H, LATENT_DIM), dev)
    if lse is not None:
        _require(lse, "lse", torch.float32, (B, S, H), dev)
        _require_contiguous(lse, "lse")
    elif return_lse:
        lse = torch.empty((B, S, H), dtype=torch.float32, device=dev)
    need = mla_decode_workspace_bytes(B, S, H, width * page_size, prefix_len)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    elif (workspace.dtype != torch.uint8 or workspace.device != dev or not workspace.is_contiguous()
          or workspace.numel() < need):
        raise ValueError(f"workspace must be a contiguous uint8 tensor of at least {need} bytes on {dev}")
    args = [_ptr(q), q.stride(0), q.stride(1), q.stride(2), _ptr(cache), pages, page_size, cache.stride(0),
            cache.stride(1)]
    if prefix_table is not None:
        args += [_ptr(prefix_table), prefix_table.shape[0], prefix_len]
    args += [_ptr(block_table), max(block_table.stride(0), width), width, _ptr(lengths), B, S, H, scale, _ptr(out),
             out.stride(0), out.stride(1), out.stride(2), _ptr(lse), _ptr(workspace), workspace.numel(),
             _stream(dev)]
    _check(fn, getattr(lib(), fn)(*args))
    if three:
        out = out.squeeze(1)
        lse = None if lse is None else lse.squeeze(1)
    return (out, lse) if return_lse else out


def mla_decode(q: torch.Tensor, cache: torch.Tensor, block_table: torch.Tensor, lengths: torch.Tensor,
               scale: float, return_lse: bool = False, out: Optional[torch.Tensor] = None,
               lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """Attention of the last S tokens of each request over its cached rows (absorbed form).

    q bf16 [B, S, H, 576] or [B, H, 576] (any strides but the last):
    the absorbed query and its rotated part.  block_table int32 [B, max_pages],
    lengths int32 [B]: rows in the cache, the S tokens' own included.
    Returns out bf16 [B, S, H, 512] (the input of the V-up product; [B, H,
    512] for a 3-D q), with ``return_lse`` also the fp32 log-sum-exp.
    ``workspace``: uint8, >= :func:`mla_decode_workspace_bytes`.
    """
    return _decode("mla_decode", q, cache, None, block_table, lengths, scale, return_lse, out, lse, workspace)


def mla_decode_shared_prefix(q: torch.Tensor, cache: torch.Tensor, prefix_table: torch.Tensor, prefix_len: int,
                             block_table: torch.Tensor, lengths: torch.Tensor, scale: float,
                             return_lse: bool = False, out: Optional[torch.Tensor] = None,
                             lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """:func:`mla_decode` where ``prefix_len`` rows (pages ``prefix_table``, int32 1-D)
    come before every request's own; they are read once for the batch.
    ``lengths`` and ``block_table`` describe the requests' own rows only."""
    return _decode("mla_decode_shared_prefix", q, cache, (prefix_table, prefix_len), block_table, lengths, scale,
                   return_lse, out, lse, workspace)


def mla_prefill(q: torch.Tensor, k_nope: torch.Tensor, k_pe: torch.Tensor, v: torch.Tensor, cu_q: torch.Tensor,
                cu_k: torch.Tensor, scale: float, causal: bool = True, return_lse: bool = False,
                out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None):
    """Attention of packed sequences over expanded keys and values.

    q bf16 [Tq, H, dn + 64], k_nope [Tk, H, dn], k_pe [Tk, 64] (shared by the
    heads), v [Tk, H, dv] with (dn, dv) = (128, 128) or (192, 256); any
    strides but the last.  Sequence b has queries cu_q[b]:cu_q[b + 1] and keys
    cu_k[b]:cu_k[b + 1] (int32 [B + 1]); with ``causal`` its queries are the
    last of its tokens.  Returns out bf16 [Tq, H, dv], with ``return_lse``
    also the fp32 log-sum-exp [Tq, H].
    """
    _require_cuda(q, "q")
    dev = q.device
    _require(v, "v", torch.bfloat16, (-1, -1, -1), dev)
    Tk, H, dv = v.shape
    dn = {128: 128, 256: 192}.get(dv)
    if dn is None:
        raise ValueError(f"v must have 128 or 256 values a head, got {dv}")
    _require(q, "q", torch.bfloat16, (-1, H, dn + ROPE_DIM), dev)
    Tq = q.shape[0]
    _require(k_nope, "k_nope", torch.bfloat16, (Tk, H, dn), dev)
    _require(k_pe, "k_pe", torch.bfloat16, (Tk, ROPE_DIM), dev)
    _require(cu_q, "cu_q", torch.int32, (-1,), dev)
    B = cu_q.shape[0] - 1
    if B < 0:
        raise ValueError("cu_q must hold at least one offset")
    _require(cu_k, "cu_k", torch.int32, (B + 1,), dev)
    _require_contiguous(cu_q, "cu_q")
    _require_contiguous(cu_k, "cu_k")
    if out is None:
        out = torch.empty((Tq, H, dv), dtype=torch.bfloat16, device=dev)
    else:
        _require(out, "out", torch.bfloat16, (Tq, H, dv), dev)
    if lse is not None:
        _require(lse, "lse", torch.float32, (Tq, H), dev)
        _require_contiguous(lse, "lse")
    elif return_lse:
        lse = torch.empty((Tq, H), dtype=torch.float32, device=dev)
    _check("mla_prefill", lib().mla_prefill(
        _ptr(q), q.stride(0), q.stride(1), _ptr(k_nope), k_nope.stride(0), k_nope.stride(1), _ptr(k_pe),
        k_pe.stride(0), _ptr(v), v.stride(0), v.stride(1), _ptr(cu_q), _ptr(cu_k), B, H, Tq, Tk, dn, dv,
        int(causal), scale, _ptr(out), out.stride(0), out.stride(1), _ptr(lse), _stream(dev)))
    return (out, lse) if return_lse else out
