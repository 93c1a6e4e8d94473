"""The feed-forward half of a layer: routing to experts, the experts' MXFP4
products, and the MXFP4 linear with an epilogue.

Same rules as the rest of the binding: every tensor is checked on the host,
outputs and the workspace are allocated with torch where they are not given,
and the HIP kernels behind the C ABI (``include/mxfp4.h``) run on the current
stream of the tensors' device.
"""

from __future__ import annotations

from functools import lru_cache
from typing import Optional, Tuple

import torch

from . import MXFP4Weight, _check, _require_bytes, _require_cuda, _require_weight, lib, weight_bytes, weight_scale_bytes
from .mla import _BF16, _F32, _I32, _addr, _raw_stream, _require

ACTIVATIONS = {"none": 0, "silu": 1, "gelu": 2, "gelu_tanh": 3, "relu": 4}
SCORINGS = {"softmax": 0, "sigmoid": 1}


def _code(table: dict, name: str, value: str) -> int:
    code = table.get(value)
    if code is None:
        raise ValueError(f"{name} must be one of {', '.join(map(repr, table))}, got {value!r}")
    return code


def _elsewhere(device: torch.device) -> bool:
    """Whether tensors on `device` need it made the current one first."""
    return device.index != torch._C._cuda_getDevice()


def moe_route(logits: torch.Tensor, top_k: int, bias: Optional[torch.Tensor] = None, scoring: str = "softmax",
              groups: int = 1, top_groups: int = 1, group_top: int = 2, renormalize: bool = True, scale: float = 1.0,
              weights: Optional[torch.Tensor] = None,
              ids: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """A token's experts: ``(weights fp32 [T, top_k], ids int32 [T, top_k])``, the best first.

    logits bf16 or fp32 [T, E] (unit stride along E); ``bias`` fp32 [E] is
    added to the scores (``scoring`` "softmax" or "sigmoid") for the choice
    only.  With ``groups`` > 1 the experts are that many runs of equal length,
    of which the ``top_groups`` best by the sum of their ``group_top`` (1 or
    2) best stay.  The weights are the chosen scores, divided by their sum if
    ``renormalize``, times ``scale``.  A logit (or bias) that is -inf or NaN
    takes its expert out; where fewer than top_k are left the ids end with -1
    and the weights with 0.
    """
    _require_cuda(logits, "logits")
    dev = logits.device
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return moe_route(logits, top_k, bias, scoring, groups, top_groups, group_top, renormalize, scale, weights,
                             ids)
    kind = logits.dtype
    if kind is not _F32 and kind is not _BF16:
        raise ValueError(f"logits must be torch.float32 or torch.bfloat16, got {kind}")
    if logits.dim() != 2 or logits.stride(1) != 1:
        _require(logits, "logits", kind, (-1, -1), dev)
    T, E = logits.shape
    if bias is not None:
        _require(bias, "bias", _F32, (E,), dev)
    if weights is None:
        weights, ldw = torch.empty_strided((T, top_k), (top_k, 1), dtype=_F32, device=dev), top_k
    else:
        ldw = _require(weights, "weights", _F32, (T, top_k), dev)[0]
    if ids is None:
        ids, ldi = torch.empty_strided((T, top_k), (top_k, 1), dtype=_I32, device=dev), top_k
    else:
        ldi = _require(ids, "ids", _I32, (T, top_k), dev)[0]
    status = lib().moe_route(
        logits.data_ptr(), logits.stride(0), 1 if kind is _F32 else 0, _addr(bias), T, E, top_k,
        _code(SCORINGS, "scoring", scoring), groups, top_groups, group_top, 1 if renormalize else 0, scale,
        weights.data_ptr(), ldw, ids.data_ptr(), ldi, _raw_stream(dev))
    if status:
        _check("moe_route", status)
    return weights, ids


# Sizes are functions of the shapes alone and asked for once per shape (a call
# through ctypes costs a microsecond).
_weight_bytes = lru_cache(maxsize=256)(lambda batch, N, K: (weight_bytes(batch, N, K), weight_scale_bytes(batch, N, K)))
_moe_bytes = lru_cache(maxsize=1024)(lambda *shape: int(lib().mxfp4_moe_workspace_bytes(*shape)))
_U8 = torch.uint8


def _weight_ok(w: torch.Tensor, ws: torch.Tensor, batch: int, N: int, K: int, dev: torch.device) -> bool:
    data, scales = _weight_bytes(batch, N, K)
    return (w.dtype is _U8 and w.device == dev and w.is_contiguous() and w.numel() >= data > 0
            and ws.dtype is _U8 and ws.device == dev and ws.is_contiguous() and ws.numel() >= scales)


def _rows_ok(t: torch.Tensor, dtype: torch.dtype, T: int, n: int, dev: torch.device) -> bool:
    return t.dtype is dtype and t.device == dev and t.shape == (T, n) and (t.stride(1) == 1 or n == 1)


def mxfp4_moe_workspace_bytes(T: int, top_k: int, experts: int, hidden: int, inner: int) -> int:
    return int(lib().mxfp4_moe_workspace_bytes(T, top_k, experts, hidden, inner))


def _workspace(workspace: Optional[torch.Tensor], need: int, dev: torch.device):
    """(tensor to keep alive, its address, its bytes)"""
    if workspace is None:
        workspace = torch.empty_strided((need,), (1,), dtype=_U8, device=dev) if need else None
    else:
        _require_bytes(workspace, "workspace", need, dev)
    return workspace, _addr(workspace), 0 if workspace is None else workspace.numel()


def mxfp4_moe(x: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, up: MXFP4Weight, down: MXFP4Weight,
              up_bias: Optional[torch.Tensor] = None, down_bias: Optional[torch.Tensor] = None,
              activation: str = "silu", gated: bool = True, residual: Optional[torch.Tensor] = None,
              out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """bf16 [T, hidden]: the chosen experts' products, weighted, plus ``residual``.

    x bf16 [T, hidden]; ids int32 and weights fp32 [T, k] (as
    :func:`moe_route` gives them); ``up`` of ``batch`` experts with 2 * inner
    rows, gate first (inner rows if not ``gated``), and ``down`` from inner
    back to hidden (:func:`quantize_weight` of a 3-D tensor, or
    :func:`mxfp4_preshuffle_weight` with ``batch``).  Per token and choice:
    x is quantised, multiplied, activated (act(gate) * up), rounded to bf16,
    quantised, multiplied, weighted and added in fp32 in the order of the
    choices.  ids outside [0, experts) add nothing.  ``up_bias`` bf16
    [experts, up.N], ``down_bias`` bf16 [experts, hidden]; ``residual`` bf16
    [T, hidden], ``out`` itself allowed.
    """
    _require_cuda(x, "x")
    dev = x.device
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return mxfp4_moe(x, ids, weights, up, down, up_bias, down_bias, activation, gated, residual, out, workspace)
    E, H, I = up.batch, up.K, down.K
    if down.batch != E or down.N != H or up.N != (2 * I if gated else I):
        raise ValueError(f"up [{E}, {up.N}, {H}] and down [{down.batch}, {down.N}, {I}] are not the two weights of "
                         f"{'gated ' if gated else ''}experts")
    T = x.shape[0]
    k = ids.shape[1] if ids.dim() == 2 else -1
    if not (_rows_ok(x, _BF16, T, H, dev) and _rows_ok(ids, _I32, T, k, dev) and _rows_ok(weights, _F32, T, k, dev)
            and _weight_ok(up.w_pre, up.ws_pre, E, up.N, H, dev) and _weight_ok(down.w_pre, down.ws_pre, E, H, I, dev)):
        _require(x, "x", _BF16, (-1, H), dev)
        _require(ids, "ids", _I32, (T, -1), dev)
        _require(weights, "weights", _F32, (T, k), dev)
        _require_weight(up.w_pre, up.ws_pre, up.N, H, dev, batch=E)
        _require_weight(down.w_pre, down.ws_pre, H, I, dev, batch=E)
    ldx, ldi, ldw = x.stride(0), ids.stride(0), weights.stride(0)
    for bias, name, n in ((up_bias, "up_bias", up.N), (down_bias, "down_bias", H)):
        if bias is not None:
            _require(bias, name, _BF16, (E, n), dev)
            if not bias.is_contiguous():
                raise ValueError(f"{name} must be contiguous")
    ldr = 0 if residual is None else _require(residual, "residual", _BF16, (T, H), dev)[0]
    if out is None:
        out, ldo = torch.empty_strided((T, H), (H, 1), dtype=_BF16, device=dev), H
    else:
        ldo = _require(out, "out", _BF16, (T, H), dev)[0]
    code = _code(ACTIVATIONS, "activation", activation)
    need = _moe_bytes(T, k, E, H, I)
    workspace, work, size = _workspace(workspace, need, dev)
    status = lib().mxfp4_moe(
        x.data_ptr(), ldx, ids.data_ptr(), ldi, weights.data_ptr(), ldw, up.w_pre.data_ptr(), up.ws_pre.data_ptr(),
        _addr(up_bias), down.w_pre.data_ptr(), down.ws_pre.data_ptr(), _addr(down_bias), _addr(residual), ldr,
        out.data_ptr(), ldo, T, k, E, H, I, code, 1 if gated else 0, work, size, _raw_stream(dev))
    if status:
        _check("mxfp4_moe", status)
    return out


def mxfp4_linear_act_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(lib().mxfp4_linear_act_workspace_bytes(M, N, K))


def mxfp4_linear_act(x: torch.Tensor, w_pre: torch.Tensor, ws_pre: torch.Tensor, N: int,
                     bias: Optional[torch.Tensor] = None, activation: str = "none", gated: bool = False,
                     residual: Optional[torch.Tensor] = None, out_dtype: torch.dtype = _BF16,
                     out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """round(act(v) + residual) of v = dq(Q(x)) dq(W)^T + bias, from bf16 x [M, K].

    ``gated``: the weight's first N/2 rows are the gate, the others what it
    multiplies: round(act(v[:, :N/2]) * v[:, N/2:] + residual).  ``residual``
    bf16, of the output's shape (``out`` itself allowed).  Otherwise as
    :func:`mxfp4_linear`.
    """
    _require_cuda(x, "x")
    dev = x.device
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return mxfp4_linear_act(x, w_pre, ws_pre, N, bias, activation, gated, residual, out_dtype, out, workspace)
    ldx = _require(x, "x", _BF16, (-1, -1), dev)[0]
    M, K = x.shape
    if gated and N % 32:
        raise ValueError(f"a gated weight has a multiple of 32 rows, got {N}")
    cols = N // 2 if gated else N
    if not _weight_ok(w_pre, ws_pre, 1, N, K, dev):
        _require_weight(w_pre, ws_pre, N, K, dev)
    if bias is not None:
        _require(bias, "bias", _BF16, (N,), dev)
    ldr = 0 if residual is None else _require(residual, "residual", _BF16, (M, cols), dev)[0]
    if out_dtype is not _BF16 and out_dtype is not _F32:
        raise ValueError(f"out_dtype must be torch.bfloat16 or torch.float32, got {out_dtype}")
    if out is None:
        out, ldo = torch.empty_strided((M, cols), (cols, 1), dtype=out_dtype, device=dev), cols
    else:
        ldo = _require(out, "out", out_dtype, (M, cols), dev)[0]
    code = _code(ACTIVATIONS, "activation", activation)
    need = int(lib().mxfp4_linear_act_workspace_bytes(M, N, K))
    workspace, work, size = _workspace(workspace, need, dev)
    status = lib().mxfp4_linear_act(
        x.data_ptr(), ldx, w_pre.data_ptr(), ws_pre.data_ptr(), _addr(bias), code, 1 if gated else 0, _addr(residual),
        ldr, out.data_ptr(), ldo, 1 if out_dtype is _F32 else 0, M, N, K, work, size, _raw_stream(dev))
    if status:
        _check("mxfp4_linear_act", status)
    return out
