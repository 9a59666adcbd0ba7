"""The routed-expert operators around the experts' LoRA: routing, the
expert-sorted rows, MXFP4 quantisation and products, and the weighted sum
back to tokens.

As in the package's other functions, arguments are marshalled to the C ABI of
include/lora_mi355x.h on torch's current stream and the computation runs in
the HIP kernels; invalid arguments raise LoraError before anything is
enqueued. Outputs are allocated from torch unless they are passed in.
"""
from __future__ import annotations

from collections import namedtuple
from typing import Optional

from . import LoraError, _check, _dev, _dtype_code, _i32, _ptr, _stream, lib

MXFP4 = namedtuple("MXFP4", ["codes", "scales"])
MXFP4.__doc__ = """Rows of K values in 4-bit floating point with a scale per 32 of them:
codes uint8 [..., K / 2], scales uint8 [..., K / 32 rounded up to a multiple of 4]."""

Routing = namedtuple("Routing", ["ids", "weights"])
Routing.__doc__ = """The experts of each token, int32 [T, top_k], and their weights, float32."""

ExpertRows = namedtuple("ExpertRows", ["row_token", "positions", "offsets", "row_slot"])
ExpertRows.__doc__ = """The choices of a routed batch sorted by expert: each row's token, each
choice's row [T, top_k], the experts' bounds and each row's adapter slot (or None)."""

_SCORES = {"softmax": 0, "sigmoid": 1}
_GROUP_SCORES = {"max": 0, "sum2": 1}


def _empty(shape, dtype, dev):
    import torch
    return torch.empty(shape, dtype=dtype, device=dev)


def _given(t, shape, dtype, what):
    """A caller's output tensor, checked."""
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype:
        raise LoraError(f"{what} must be {dtype} {tuple(shape)}")
    return t


def route_experts(logits, top_k: int, *, scores: str = "softmax", bias=None, groups: int = 1,
                  top_groups: Optional[int] = None, group_score: str = "max",
                  renormalize: bool = True, scaling: float = 1.0,
                  out: Optional[Routing] = None) -> Routing:
    """The top_k experts of each token of logits [T, experts] and their weights.

    Scores are softmax or sigmoid of the logits; bias (float32 [experts])
    counts for the choice alone, not for the weights. With top_groups < groups
    only the experts of a token's best groups of consecutive ones are open to
    it (a group is worth its best expert, or the sum of its two best). Ties go
    to the lowest index; a NaN or -inf logit closes an expert, and a token
    with fewer than top_k open experts gets id -1 and weight 0 for the rest.
    Weights are divided by their sum (renormalize) and multiplied by scaling."""
    import torch
    if scores not in _SCORES or group_score not in _GROUP_SCORES:
        raise LoraError("scores must be softmax or sigmoid, group_score max or sum2")
    dev = _dev(logits, bias)
    if logits.dim() != 2:
        raise LoraError("logits must be [T, experts]")
    T, E = logits.shape
    if bias is not None and (bias.dtype != torch.float32 or bias.numel() != E):
        raise LoraError("bias must be float32 [experts]")
    if out is None:
        out = Routing(_empty((T, top_k), torch.int32, dev), _empty((T, top_k), torch.float32, dev))
    else:
        _given(out.ids, (T, top_k), torch.int32, "ids")
        _given(out.weights, (T, top_k), torch.float32, "weights")
        _dev(logits, *out)
    st = lib().lora_route_experts(_dtype_code(logits), logits.data_ptr(), T, E, top_k,
                                  _SCORES[scores], _ptr(bias), groups,
                                  groups if top_groups is None else top_groups,
                                  _GROUP_SCORES[group_score], int(renormalize), scaling,
                                  out.ids.data_ptr(), out.weights.data_ptr(), _stream(dev))
    _check(st, "lora_route_experts")
    return out


def expert_rows(ids, num_experts: int, token_slot=None) -> ExpertRows:
    """Sort the choices ids [T, top_k] by expert: one row per choice, stably,
    choices outside [0, num_experts) after every expert's. With token_slot
    [T], each row's adapter slot as well (what apply_linear_from_experts_
    takes, with offsets)."""
    import torch
    ids = _i32(ids)
    if token_slot is not None:
        token_slot = _i32(token_slot)
    dev = _dev(ids, token_slot)
    if ids.dim() != 2:
        raise LoraError("ids must be [T, top_k]")
    T, k = ids.shape
    if token_slot is not None and token_slot.numel() != T:
        raise LoraError("token_slot must be [T]")
    n = T * k
    row_token = _empty((n,), torch.int32, dev)
    positions = _empty((T, k), torch.int32, dev)
    offsets = _empty((num_experts + 1,), torch.int32, dev)
    row_slot = None if token_slot is None else _empty((n,), torch.int32, dev)
    L = lib()
    nws = int(L.lora_expert_rows_workspace_bytes(T, k, num_experts))
    ws = _empty((nws,), torch.uint8, dev) if nws else None
    st = L.lora_expert_rows(ids.data_ptr(), T, k, num_experts, _ptr(token_slot),
                            row_token.data_ptr(), positions.data_ptr(), offsets.data_ptr(),
                            _ptr(row_slot), _ptr(ws), nws, _stream(dev))
    _check(st, "lora_expert_rows")
    return ExpertRows(row_token, positions, offsets, row_slot)


def combine_experts(rows, positions, weights, *, residual=None, y=None):
    """y[t] = residual[t] + sum over j of weights[t, j] * rows[positions[t, j]]
    in float32, rounded once; positions outside the rows add nothing. residual
    may be y itself (an in-place sum)."""
    import torch
    positions = _i32(positions)
    dev = _dev(rows, positions, weights, residual, y)
    if positions.dim() != 2 or rows.dim() != 2:
        raise LoraError("rows must be [num_rows, width] and positions [T, top_k]")
    T, k = positions.shape
    n, width = rows.shape
    _given(weights, (T, k), torch.float32, "weights")
    if residual is not None:
        _given(residual, (T, width), rows.dtype, "residual")
    if y is None:
        y = _empty((T, width), rows.dtype, dev)
    else:
        _given(y, (T, width), rows.dtype, "y")
    st = lib().lora_combine_experts(_dtype_code(rows), rows.data_ptr(), n, width,
                                    positions.data_ptr(), weights.data_ptr(), T, k,
                                    _ptr(residual), y.data_ptr(), _stream(dev))
    _check(st, "lora_combine_experts")
    return y


def _scale_row(K: int) -> int:
    return (K // 32 + 3) // 4 * 4


def _quantize(form, x, row_index, lead, rows, K):
    import torch
    dev = _dev(x, row_index)
    codes = _empty((*lead, K // 2), torch.uint8, dev)
    scales = _empty((*lead, _scale_row(K)), torch.uint8, dev)
    rows_out = None if form == 0 else _empty((rows, K), x.dtype, dev)
    x_rows = x.shape[0] if form else rows
    st = lib().lora_quantize_mxfp4(_dtype_code(x), form, x.data_ptr(), x_rows, _ptr(row_index),
                                   rows, K, _ptr(rows_out), codes.data_ptr(), scales.data_ptr(),
                                   _stream(dev))
    _check(st, "lora_quantize_mxfp4")
    return rows_out, MXFP4(codes, scales)


def quantize_mxfp4(x) -> MXFP4:
    """x [..., K] (bf16 or float32, K a multiple of 32) in MXFP4: per 32
    values a power-of-two scale from the largest of them, and the nearest
    4-bit values. A block that holds a NaN or an infinity becomes NaN."""
    if x.dim() < 1 or x.shape[-1] < 1:
        raise LoraError("x must be [..., K]")
    K = x.shape[-1]
    return _quantize(0, x, None, tuple(x.shape[:-1]), x.numel() // K, K)[1]


def gather_quantize_mxfp4(x, row_token):
    """The rows x[row_token] (an expert-sorted batch from its tokens), as they
    are and in MXFP4: (rows, MXFP4). Indices are clamped to x's rows."""
    row_token = _i32(row_token)
    if x.dim() != 2 or row_token.dim() != 1:
        raise LoraError("x must be [T, K] and row_token [rows]")
    n, K = row_token.numel(), x.shape[1]
    return _quantize(1, x, row_token, (n,), n, K)


def silu_mul_quantize_mxfp4(gate_up):
    """silu(gate) * up of gate_up [rows, 2 K] (gate in the first K columns),
    in gate_up's type and in MXFP4: (rows, MXFP4)."""
    if gate_up.dim() != 2 or gate_up.shape[1] % 2:
        raise LoraError("gate_up must be [rows, 2 K]")
    n, K = gate_up.shape[0], gate_up.shape[1] // 2
    return _quantize(2, gate_up, None, (n,), n, K)


def _held(q: MXFP4, what: str):
    """Rows and K of an MXFP4 pair, checked."""
    import torch
    codes, scales = q
    K = codes.shape[-1] * 2
    if (codes.dtype != torch.uint8 or scales.dtype != torch.uint8
            or tuple(scales.shape) != (*codes.shape[:-1], _scale_row(K))):
        raise LoraError(f"{what}: codes must be uint8 [..., K / 2] and scales uint8 "
                        "[..., K / 32 rounded up to a multiple of 4]")
    return K


def dequantize_mxfp4(q: MXFP4, dtype=None):
    """The values an MXFP4 pair stands for, in dtype (bf16 unless given)."""
    import torch
    K = _held(q, "dequantize_mxfp4")
    dev = _dev(*q)
    out = _empty((*q.codes.shape[:-1], K), dtype or torch.bfloat16, dev)
    st = lib().lora_dequantize_mxfp4(_dtype_code(out), q.codes.data_ptr(), q.scales.data_ptr(),
                                     out.numel() // max(K, 1), K, out.data_ptr(), _stream(dev))
    _check(st, "lora_dequantize_mxfp4")
    return out


def _product(x, w, offsets, dtype, y, what):
    import torch
    dev = _dev(*x, *w, offsets, y)
    K = _held(x, "x")
    if _held(w, "w") != K or x.codes.dim() != 2:
        raise LoraError(f"{what}: shape mismatch between x and w")
    rows, N = x.codes.shape[0], w.codes.shape[-2]
    if y is None:
        y = _empty((rows, N), dtype or torch.bfloat16, dev)
    else:
        _given(y, (rows, N), dtype or y.dtype, "y")
    return dev, rows, N, K, y


def mxfp4_linear(x: MXFP4, w: MXFP4, *, dtype=None, y=None):
    """y = x @ w^T for x [rows, K] and w [N, K] in MXFP4 (w: the shards of a
    fused projection stacked along N), accumulated in float32; y is bf16
    unless dtype or y says float32. A target's LoRA delta goes onto y with
    apply_linear_."""
    dev, rows, N, K, y = _product(x, w, None, dtype, y, "mxfp4_linear")
    if w.codes.dim() != 2:
        raise LoraError("mxfp4_linear: w must be [N, K]")
    st = lib().lora_mxfp4_linear(_dtype_code(y), x.codes.data_ptr(), x.scales.data_ptr(), rows,
                                 w.codes.data_ptr(), w.scales.data_ptr(), N, K, y.data_ptr(),
                                 _stream(dev))
    _check(st, "lora_mxfp4_linear")
    return y


def mxfp4_expert_linear(x: MXFP4, w: MXFP4, offsets, *, dtype=None, y=None):
    """Each row of the expert-sorted x [rows, K] against its expert's weight
    of w [experts, N, K], offsets [experts + 1] the experts' bounds; rows
    outside them become 0. The experts' LoRA goes onto y with
    apply_linear_from_experts_."""
    offsets = _i32(offsets)
    dev, rows, N, K, y = _product(x, w, offsets, dtype, y, "mxfp4_expert_linear")
    if w.codes.dim() != 3 or offsets.numel() != w.codes.shape[0] + 1:
        raise LoraError("mxfp4_expert_linear: w must be [experts, N, K], offsets [experts + 1]")
    st = lib().lora_mxfp4_expert_linear(_dtype_code(y), x.codes.data_ptr(), x.scales.data_ptr(),
                                        rows, w.codes.data_ptr(), w.scales.data_ptr(), N, K,
                                        offsets.data_ptr(), w.codes.shape[0], y.data_ptr(),
                                        _stream(dev))
    _check(st, "lora_mxfp4_expert_linear")
    return y
