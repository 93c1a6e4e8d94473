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

from . import _check, _require_cuda, lib

LATENT_DIM = 512
ROPE_DIM = 64
ROW_DIM = LATENT_DIM + ROPE_DIM


# These calls run once per layer and decoding step, where a call's time on the
# host is the call's time.  So each first asks one written-out question, whether
# everything is as it should be, and only where it is not goes through the
# tensors one by one to name what is wrong; device addresses go to ctypes as
# plain integers, and the stream's handle is asked for without building a
# stream object.  (61 tokens appended: 19.8 -> 9.8 us a call.)

_BF16, _F32, _I32, _I64 = torch.bfloat16, torch.float32, torch.int32, torch.int64

def _require(t: torch.Tensor, name: str, dtype: torch.dtype, shape, device: torch.device):
    """t has this dtype and shape (-1: any size) on `device` and unit stride
    along its last dimension; returns its strides."""
    size, strides = t.shape, t.stride()
    ok = t.dtype is dtype and t.device == device and len(size) == len(shape)
    if ok:
        for n, w in zip(size, shape):
            if n != w and w >= 0:
                ok = False
    if not ok:
        want = ", ".join("any" if w < 0 else str(w) for w in shape)
        raise ValueError(f"{name} must be {dtype} [{want}] on {device}, got {t.dtype} {tuple(size)} on {t.device}")
    if strides[-1] != 1 and size[-1] > 1 and t.numel():
        raise ValueError(f"{name} must have unit stride along its last dimension")
    return strides


def _require_contiguous(t: torch.Tensor, name: str) -> None:
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _addr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _raw_stream(device: torch.device) -> int:
    return torch._C._cuda_getCurrentRawStream(device.index)


def mla_decode_workspace_bytes(B: int, S: int, H: int, max_tokens: int, prefix_len: int = 0) -> int:
    return int(lib().mla_decode_workspace_bytes(B, S, H, max_tokens, prefix_len))


def set_mla_rows(rows: int) -> None:
    """Test hook (include/mxfp4_testing.h), for the calling thread only: query
    rows per workgroup of the decode kernels (16, 32, 128; 0 = by size)."""
    _check("mla_testing_set_rows", lib().mla_testing_set_rows(rows))


def set_mla_prefill_rows(rows: int) -> None:
    """Test hook (include/mxfp4_testing.h), for the calling thread only: query
    rows per workgroup of the prefill kernels (32, 128; 0 = by size)."""
    _check("mla_testing_set_prefill_rows", lib().mla_testing_set_prefill_rows(rows))


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
    itself, or the last 64 columns of an absorbed query).  Nothing is written
    for a token whose position lies outside the table: its rows of an allocated
    ``q_out`` are not initialised.
    """
    _require_cuda(kv, "kv")
    dev = kv.device
    H = 0
    rotated = (None, 0, 0, None, 0, 0)
    T, width = kv.shape
    pages, page_size, row = cache.shape
    kv_strides, cache_strides = kv.stride(), cache.stride()
    if not (width == ROW_DIM == row and kv.dtype is _BF16 and kv_strides[1] == 1
            and cache.dtype is _BF16 and cache.device == dev and cache_strides[2] == 1
            and norm_weight.dtype is _BF16 and norm_weight.device == dev and norm_weight.shape == (LATENT_DIM,)
            and norm_weight.stride(0) == 1
            and slots.dtype is _I64 and slots.device == dev and slots.shape == (T,) and slots.stride(0) == 1
            and positions.dtype is _I64 and positions.device == dev and positions.shape == (T,)
            and positions.stride(0) == 1
            and cos_sin.dtype is _F32 and cos_sin.device == dev and cos_sin.dim() == 2
            and cos_sin.shape[1] == ROPE_DIM and cos_sin.is_contiguous()):
        _require(kv, "kv", _BF16, (-1, ROW_DIM), dev)
        _require(norm_weight, "norm_weight", _BF16, (LATENT_DIM,), dev)
        _require(cache, "cache", _BF16, (-1, -1, ROW_DIM), dev)
        _require(slots, "slots", _I64, (T,), dev)
        _require(positions, "positions", _I64, (T,), dev)
        _require(cos_sin, "cos_sin", _F32, (-1, ROPE_DIM), dev)
        _require_contiguous(cos_sin, "cos_sin")
    if q_pe is not None:
        q_strides = _require(q_pe, "q_pe", _BF16, (T, -1, ROPE_DIM), dev)
        H = q_pe.shape[1]
        if q_out is None:
            q_out = torch.empty((T, H, ROPE_DIM), dtype=_BF16, device=dev)
        o_strides = _require(q_out, "q_out", _BF16, (T, H, ROPE_DIM), dev)
        if H:
            rotated = (q_pe.data_ptr(), q_strides[0], q_strides[1], q_out.data_ptr(), o_strides[0], o_strides[1])
    elif q_out is not None:
        raise ValueError("q_out is given without q_pe")
    status = lib().mla_cache_append(
        kv.data_ptr(), kv_strides[0], norm_weight.data_ptr(), eps, cos_sin.data_ptr(), cos_sin.shape[0],
        positions.data_ptr(), slots.data_ptr(), 1 if interleaved else 0, *rotated, cache.data_ptr(), pages, page_size,
        cache_strides[0], cache_strides[1], T, H, _raw_stream(dev))
    if status:
        _check("mla_cache_append", status)
    return q_out


def _decode(fn, q, cache, prefix, block_table, lengths, scale, return_lse, out, lse, workspace):
    _require_cuda(q, "q")
    dev = q.device
    three = q.dim() == 3
    if three:
        q = q.unsqueeze(1)
        out = None if out is None else out.unsqueeze(1)
        lse = None if lse is None else lse.unsqueeze(1)
    if q.dim() != 4 or cache.dim() != 3 or block_table.dim() != 2:
        raise ValueError("q must have 3 or 4 dimensions, cache 3 and block_table 2")
    B, S, H, row = q.shape
    pages, page_size, cache_dim = cache.shape
    requests, width = block_table.shape
    q_strides, cache_strides, table_strides = q.stride(), cache.stride(), block_table.stride()
    if not (row == ROW_DIM == cache_dim and q.dtype is _BF16 and q_strides[3] == 1
            and cache.dtype is _BF16 and cache.device == dev and cache_strides[2] == 1
            and block_table.dtype is _I32 and block_table.device == dev and requests == B and table_strides[1] == 1
            and lengths.dtype is _I32 and lengths.device == dev and lengths.shape == (B,)
            and lengths.is_contiguous()):
        _require(q, "q", _BF16, (-1, -1, -1, ROW_DIM), dev)
        _require(cache, "cache", _BF16, (-1, -1, ROW_DIM), dev)
        _require(block_table, "block_table", _I32, (B, -1), dev)
        _require(lengths, "lengths", _I32, (B,), dev)
        _require_contiguous(lengths, "lengths")
    # (One request's row stride means nothing.)
    ldt = table_strides[0] if B > 1 else width
    if 0 < ldt < width:
        raise ValueError("block_table's rows may be one row for all requests (stride 0), but must not overlap in "
                         f"part: row stride {ldt}, width {width}")
    shared, prefix_len = (), 0
    if prefix is not None:
        prefix_table, prefix_len = prefix
        _require(prefix_table, "prefix_table", _I32, (-1,), dev)
        _require_contiguous(prefix_table, "prefix_table")
        prefix_pages = prefix_table.shape[0]
        if not 0 <= prefix_len <= prefix_pages * page_size:
            raise ValueError(f"prefix_len {prefix_len} does not fit prefix_table's {prefix_pages} pages")
        shared = (prefix_table.data_ptr(), prefix_pages, prefix_len)
    if out is None:
        out = torch.empty((B, S, H, LATENT_DIM), dtype=_BF16, device=dev)
        out_strides = out.stride()
    else:
        out_strides = _require(out, "out", _BF16, (B, S, H, LATENT_DIM), dev)
    if lse is not None:
        _require(lse, "lse", _F32, (B, S, H), dev)
        _require_contiguous(lse, "lse")
    elif return_lse:
        lse = torch.empty((B, S, H), dtype=_F32, device=dev)
    handle = lib()
    need = handle.mla_decode_workspace_bytes(B, S, H, width * page_size, prefix_len)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    else:
        _require(workspace, "workspace", torch.uint8, (-1,), dev)
        _require_contiguous(workspace, "workspace")
        if workspace.shape[0] < need:
            raise ValueError(f"workspace holds {workspace.shape[0]} bytes, {need} needed")
    status = getattr(handle, fn)(
        q.data_ptr(), q_strides[0], q_strides[1], q_strides[2], cache.data_ptr(), pages, page_size, cache_strides[0],
        cache_strides[1], *shared, block_table.data_ptr(), ldt, width, lengths.data_ptr(),
        B, S, H, scale, out.data_ptr(), out_strides[0], out_strides[1], out_strides[2], _addr(lse),
        workspace.data_ptr(), workspace.shape[0], _raw_stream(dev))
    if status:
        _check(fn, status)
    if three:
        out = out.squeeze(1)
        lse = None if lse is None else lse.squeeze(1)
    return (out, lse) if return_lse else out


def mla_decode(q: torch.Tensor, cache: torch.Tensor, block_table: torch.Tensor, lengths: torch.Tensor,
               scale: float, return_lse: bool = False, out: Optional[torch.Tensor] = None,
               lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """Attention of the last S tokens of each request over its cached rows (absorbed form).

    q bf16 [B, S, H, 576] or [B, H, 576] (any strides but the last):
    the absorbed query and its rotated part.  block_table int32 [B, max_pages]
    (one row ``expand``ed over requests that share their pages is read as it
    is), lengths int32 [B]: rows in the cache, the S tokens' own included.
    Returns out bf16 [B, S, H, 512] (the input of the V-up product; [B, H,
    512] for a 3-D q), with ``return_lse`` also the fp32 log-sum-exp.
    ``workspace``: uint8, >= :func:`mla_decode_workspace_bytes`.  The table's
    width, not the lengths, chooses the kernel's row blocks: a narrow view of a
    wide table (``table[:, :pages_in_use]``) is faster where requests are short.
    """
    return _decode("mla_decode", q, cache, None, block_table, lengths, scale, return_lse, out, lse, workspace)


def mla_decode_shared_prefix(q: torch.Tensor, cache: torch.Tensor, prefix_table: torch.Tensor, prefix_len: int,
                             block_table: torch.Tensor, lengths: torch.Tensor, scale: float,
                             return_lse: bool = False, out: Optional[torch.Tensor] = None,
                             lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """:func:`mla_decode` where ``prefix_len`` rows (pages ``prefix_table``, int32 1-D)
    come before every request's own; they are read for the batch together.
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
    if q.dim() != 3 or k_nope.dim() != 3 or k_pe.dim() != 2 or v.dim() != 3 or cu_q.dim() != 1:
        raise ValueError("q, k_nope and v must have 3 dimensions, k_pe 2 and cu_q 1")
    Tk, H, dv = v.shape
    dn = 128 if dv == 128 else 192 if dv == 256 else 0
    if not dn:
        raise ValueError(f"v must have 128 or 256 values a head, got {dv}")
    Tq = q.shape[0]
    B = cu_q.shape[0] - 1
    if B < 0:
        raise ValueError("cu_q must hold at least one offset")
    q_strides, k_strides, pe_strides, v_strides = q.stride(), k_nope.stride(), k_pe.stride(), v.stride()
    if not (q.dtype is _BF16 and q.shape == (Tq, H, dn + ROPE_DIM) and q_strides[2] == 1
            and k_nope.dtype is _BF16 and k_nope.device == dev and k_nope.shape == (Tk, H, dn) and k_strides[2] == 1
            and k_pe.dtype is _BF16 and k_pe.device == dev and k_pe.shape == (Tk, ROPE_DIM) and pe_strides[1] == 1
            and v.dtype is _BF16 and v.device == dev and v_strides[2] == 1
            and cu_q.dtype is _I32 and cu_q.device == dev and cu_q.is_contiguous()
            and cu_k.dtype is _I32 and cu_k.device == dev and cu_k.shape == (B + 1,) and cu_k.is_contiguous()):
        _require(v, "v", _BF16, (-1, -1, -1), dev)
        _require(q, "q", _BF16, (-1, H, dn + ROPE_DIM), dev)
        _require(k_nope, "k_nope", _BF16, (Tk, H, dn), dev)
        _require(k_pe, "k_pe", _BF16, (Tk, ROPE_DIM), dev)
        _require(cu_q, "cu_q", _I32, (-1,), dev)
        _require(cu_k, "cu_k", _I32, (B + 1,), dev)
        _require_contiguous(cu_q, "cu_q")
        _require_contiguous(cu_k, "cu_k")
    if out is None:
        out = torch.empty((Tq, H, dv), dtype=_BF16, device=dev)
        out_strides = out.stride()
    else:
        out_strides = _require(out, "out", _BF16, (Tq, H, dv), dev)
    if lse is not None:
        _require(lse, "lse", _F32, (Tq, H), dev)
        _require_contiguous(lse, "lse")
    elif return_lse:
        lse = torch.empty((Tq, H), dtype=_F32, device=dev)
    status = lib().mla_prefill(
        q.data_ptr(), q_strides[0], q_strides[1], k_nope.data_ptr(), k_strides[0], k_strides[1], k_pe.data_ptr(),
        pe_strides[0], v.data_ptr(), v_strides[0], v_strides[1], cu_q.data_ptr(), cu_k.data_ptr(), B, H, Tq, Tk, dn,
        dv, 1 if causal else 0, scale, out.data_ptr(), out_strides[0], out_strides[1], _addr(lse), _raw_stream(dev))
    if status:
        _check("mla_prefill", status)
    return (out, lse) if return_lse else out
