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

from . import LoraError, _check, _dtype_code, _i32, lib

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

# A decode step's operators take less time on the GPU than their calls take on
# the host (3.4 us for the launch by way of ctypes), so the helpers below do
# their checks without building shapes, devices or streams.
_T = None


def _torch():
    global _T
    if _T is None:
        import torch
        _T = torch
    return _T


def _gpu(*tensors):
    """The device of contiguous tensors (None is skipped), checked."""
    dev = None
    for t in tensors:
        if t is None:
            continue
        if not t.is_cuda:
            raise LoraError("all tensors must be on the GPU (no CPU fallback)")
        if not t.is_contiguous():
            raise LoraError("tensors must be contiguous")
        if dev is None:
            dev = t.get_device()
        elif t.get_device() != dev:
            raise LoraError("tensors on different devices")
    return dev


def _stream(dev: int) -> int:
    raw = getattr(_T._C, "_cuda_getCurrentRawStream", None)
    return raw(dev) if raw else _T.cuda.current_stream(dev).cuda_stream


def _new(n, m, dtype, dev):
    return _T.empty_strided((n, m), (m, 1), dtype=dtype, device=dev)


def _new1(n, dtype, dev):
    return _T.empty_strided((n,), (1,), dtype=dtype, device=dev)


def _given(t, n, m, dtype, what):
    """A caller's [n, m] tensor, checked."""
    if t.dim() != 2 or t.shape[0] != n or t.shape[1] != m or t.dtype != dtype:
        raise LoraError(f"{what} must be {dtype} [{n}, {m}]")
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
    torch = _torch()
    if scores not in _SCORES or group_score not in _GROUP_SCORES:
        raise LoraError("scores must be softmax or sigmoid, group_score max or sum2")
    if logits.dim() != 2:
        raise LoraError("logits must be [T, experts]")
    T, E = logits.shape
    if bias is not None and (bias.dtype != torch.float32 or bias.numel() != E):
        raise LoraError("bias must be float32 [experts]")
    if top_k < 1:
        raise LoraError("top_k must be at least 1")
    if out is None:
        dev = _gpu(logits, bias)
        ids = _new(T, top_k, torch.int32, dev)
        weights = _new(T, top_k, torch.float32, dev)
        out = Routing(ids, weights)
    else:
        ids = _given(out.ids, T, top_k, torch.int32, "ids")
        weights = _given(out.weights, T, top_k, torch.float32, "weights")
        dev = _gpu(logits, bias, ids, weights)
    st = lib().lora_route_experts(_dtype_code(logits), logits.data_ptr(), T, E, top_k,
                                  _SCORES[scores], None if bias is None else bias.data_ptr(),
                                  groups, groups if top_groups is None else top_groups,
                                  _GROUP_SCORES[group_score], renormalize, scaling,
                                  ids.data_ptr(), weights.data_ptr(), _stream(dev))
    if st:
        _check(st, "lora_route_experts")
    return out


def expert_rows(ids, num_experts: int, token_slot=None) -> ExpertRows:
    """Sort the choices ids [T, top_k] by expert: one row per choice, stably,
    choices outside [0, num_experts) after every expert's. With token_slot
    [T], each row's adapter slot as well (what apply_linear_from_experts_
    takes, with offsets)."""
    torch = _torch()
    ids = _i32(ids)
    if token_slot is not None:
        token_slot = _i32(token_slot)
    dev = _gpu(ids, token_slot)
    if ids.dim() != 2:
        raise LoraError("ids must be [T, top_k]")
    T, k = ids.shape
    if token_slot is not None and token_slot.numel() != T:
        raise LoraError("token_slot must be [T]")
    if num_experts < 1:
        raise LoraError("num_experts must be at least 1")
    n = T * k
    i32 = torch.int32
    row_token = _new1(n, i32, dev)
    positions = _new(T, k, i32, dev)
    offsets = _new1(num_experts + 1, i32, dev)
    row_slot = None if token_slot is None else _new1(n, i32, dev)
    L = lib()
    nws = L.lora_expert_rows_workspace_bytes(T, k, num_experts)
    ws = _new1(nws, torch.uint8, dev) if nws else None
    st = L.lora_expert_rows(ids.data_ptr(), T, k, num_experts,
                            None if token_slot is None else token_slot.data_ptr(),
                            row_token.data_ptr(), positions.data_ptr(), offsets.data_ptr(),
                            None if row_slot is None else row_slot.data_ptr(),
                            None if ws is None else ws.data_ptr(), nws, _stream(dev))
    if st:
        _check(st, "lora_expert_rows")
    return ExpertRows(row_token, positions, offsets, row_slot)


def combine_experts(rows, positions, weights, *, residual=None, y=None):
    """y[t] = residual[t] + sum over j of weights[t, j] * rows[positions[t, j]]
    in float32, rounded once; positions outside the rows add nothing. residual
    may be y itself (an in-place sum)."""
    torch = _torch()
    positions = _i32(positions)
    dev = _gpu(rows, positions, weights, residual, y)
    if positions.dim() != 2 or rows.dim() != 2:
        raise LoraError("rows must be [num_rows, width] and positions [T, top_k]")
    T, k = positions.shape
    n, width = rows.shape
    _given(weights, T, k, torch.float32, "weights")
    if residual is not None:
        _given(residual, T, width, rows.dtype, "residual")
    if y is None:
        y = _new(T, width, rows.dtype, dev)
    else:
        _given(y, T, width, rows.dtype, "y")
    st = lib().lora_combine_experts(_dtype_code(rows), rows.data_ptr(), n, width,
                                    positions.data_ptr(), weights.data_ptr(), T, k,
                                    None if residual is None else residual.data_ptr(),
                                    y.data_ptr(), _stream(dev))
    if st:
        _check(st, "lora_combine_experts")
    return y


def _scale_row(K: int) -> int:
    return (K // 32 + 3) // 4 * 4


def _quantize(form, x, row_index, rows, K, x_rows):
    u8 = _torch().uint8
    dev = _gpu(x, row_index)
    codes = _new(rows, K // 2, u8, dev)
    scales = _new(rows, _scale_row(K), u8, dev)
    rows_out = None if form == 0 else _new(rows, K, x.dtype, dev)
    st = lib().lora_quantize_mxfp4(_dtype_code(x), form, x.data_ptr(), x_rows,
                                   None if row_index is None else row_index.data_ptr(), rows, K,
                                   None if form == 0 else rows_out.data_ptr(), codes.data_ptr(),
                                   scales.data_ptr(), _stream(dev))
    if st:
        _check(st, "lora_quantize_mxfp4")
    return rows_out, codes, scales


def quantize_mxfp4(x) -> MXFP4:
    """x [..., K] (bf16 or float32, K a multiple of 32) in MXFP4: per 32
    values a power-of-two scale from the largest of them, and the nearest
    4-bit values. A block that holds a NaN or an infinity becomes NaN."""
    if x.dim() < 1 or x.shape[-1] < 1:
        raise LoraError("x must be [..., K]")
    K = x.shape[-1]
    rows = x.numel() // K
    _, codes, scales = _quantize(0, x, None, rows, K, rows)
    if x.dim() != 2:
        codes = codes.view(*x.shape[:-1], K // 2)
        scales = scales.view(*x.shape[:-1], -1)
    return MXFP4(codes, scales)


def gather_quantize_mxfp4(x, row_token):
    """The rows x[row_token] (an expert-sorted batch from its tokens), as they
    are and in MXFP4: (rows, MXFP4). Indices are clamped to x's rows."""
    row_token = _i32(row_token)
    if x.dim() != 2 or row_token.dim() != 1:
        raise LoraError("x must be [T, K] and row_token [rows]")
    rows, codes, scales = _quantize(1, x, row_token, row_token.numel(), x.shape[1], x.shape[0])
    return rows, MXFP4(codes, scales)


def silu_mul_quantize_mxfp4(gate_up):
    """silu(gate) * up of gate_up [rows, 2 K] (gate in the first K columns),
    in gate_up's type and in MXFP4: (rows, MXFP4)."""
    if gate_up.dim() != 2 or gate_up.shape[1] % 2:
        raise LoraError("gate_up must be [rows, 2 K]")
    n = gate_up.shape[0]
    rows, codes, scales = _quantize(2, gate_up, None, n, gate_up.shape[1] // 2, n)
    return rows, MXFP4(codes, scales)


def _held(q: MXFP4, what: str):
    """Rows (all leading dimensions) and K of an MXFP4 pair, checked."""
    codes, scales = q
    K = codes.shape[-1] * 2
    ld = (K // 32 + 3) // 4 * 4
    rows = codes.numel() * 2 // K if K else 0
    u8 = _T.uint8
    if (codes.dtype is not u8 or scales.dtype is not u8 or scales.dim() != codes.dim()
            or scales.shape[-1] != ld or scales.numel() != rows * ld
            or (codes.dim() == 3 and scales.shape[0] != codes.shape[0])):
        raise LoraError(f"{what}: codes must be uint8 [..., K / 2] and scales uint8 "
                        "[..., K / 32 rounded up to a multiple of 4]")
    return rows, K


def dequantize_mxfp4(q: MXFP4, dtype=None):
    """The values an MXFP4 pair stands for, in dtype (bf16 unless given)."""
    torch = _torch()
    rows, K = _held(q, "dequantize_mxfp4")
    codes, scales = q
    dev = _gpu(codes, scales)
    out = _new(rows, K, dtype or torch.bfloat16, dev)
    st = lib().lora_dequantize_mxfp4(_dtype_code(out), codes.data_ptr(), scales.data_ptr(), rows,
                                     K, out.data_ptr(), _stream(dev))
    if st:
        _check(st, "lora_dequantize_mxfp4")
    return out if codes.dim() == 2 else out.view(*codes.shape[:-1], K)


def _product(x, w, offsets, dtype, y, what):
    torch = _torch()
    dev = _gpu(x[0], x[1], w[0], w[1], offsets, y)
    rows, K = _held(x, what)
    if _held(w, what)[1] != K or x[0].dim() != 2 or w[0].dim() != (2 if offsets is None else 3):
        raise LoraError(f"{what}: shape mismatch between x and w")
    N = w[0].shape[-2]
    if y is None:
        y = _new(rows, N, dtype or torch.bfloat16, dev)
    else:
        _given(y, rows, N, dtype or y.dtype, "y")
    return dev, rows, N, K, y


def mxfp4_linear(x: MXFP4, w: MXFP4, *, dtype=None, y=None):
    """y = x @ w^T for x [rows, K] and w [N, K] in MXFP4 (w: the shards of a
    fused projection stacked along N), accumulated in float32; y is bf16
    unless dtype or y says float32. A target's LoRA delta goes onto y with
    apply_linear_."""
    dev, rows, N, K, y = _product(x, w, None, dtype, y, "mxfp4_linear")
    st = lib().lora_mxfp4_linear(_dtype_code(y), x[0].data_ptr(), x[1].data_ptr(), rows,
                                 w[0].data_ptr(), w[1].data_ptr(), N, K, y.data_ptr(),
                                 _stream(dev))
    if st:
        _check(st, "lora_mxfp4_linear")
    return y


def mxfp4_expert_linear(x: MXFP4, w: MXFP4, offsets, *, dtype=None, y=None):
    """Each row of the expert-sorted x [rows, K] against its expert's weight
    of w [experts, N, K], offsets [experts + 1] the experts' bounds; rows
    outside them become 0. The experts' LoRA goes onto y with
    apply_linear_from_experts_."""
    offsets = _i32(offsets)
    dev, rows, N, K, y = _product(x, w, offsets, dtype, y, "mxfp4_expert_linear")
    E = w[0].shape[0]
    if offsets.numel() != E + 1:
        raise LoraError("mxfp4_expert_linear: offsets must be [experts + 1]")
    st = lib().lora_mxfp4_expert_linear(_dtype_code(y), x[0].data_ptr(), x[1].data_ptr(), rows,
                                        w[0].data_ptr(), w[1].data_ptr(), N, K,
                                        offsets.data_ptr(), E, y.data_ptr(), _stream(dev))
    if st:
        _check(st, "lora_mxfp4_expert_linear")
    return y
