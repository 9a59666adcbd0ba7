"""The routed-expert operators around the experts' LoRA: routing, the
expert-sorted rows, MXFP4 quantisation and products, and the weighted sum
back to tokens.

As in the package's other functions, arguments are marshalled to the C ABI of
include/lora_mi355x.h on torch's current stream and the computation runs in
the HIP kernels; invalid arguments raise LoraError before anything is
enqueued. Outputs are allocated from torch unless they are passed in. Index
tensors are int32; other types are converted first, and an int64 value that
int32 does not hold stays out of range. The marshalling is compiled
(csrc/experts/binding.cpp, built as _experts.so next to this file): a decode
step's operators take less time than such calls in Python.
"""
from __future__ import annotations

import os
from collections import namedtuple
from typing import Optional

from . import LoraError, lib

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
_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_experts.so")
_EXT = None


def _load():
    """The compiled binding (after the library, which it calls)."""
    global _EXT
    lib()
    if not os.path.exists(_PATH):
        raise LoraError(f"{_PATH} is not built: run `python -m adapter_lora_serving_amd.build`"
                        " (there is no CPU or PyTorch fallback)")
    import torch
    from . import _experts
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    _experts.setup(LoraError, raw or (lambda d: torch.cuda.current_stream(d).cuda_stream))
    _EXT = _experts
    return _EXT


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
    if scores not in _SCORES or group_score not in _GROUP_SCORES:
        raise LoraError("scores must be softmax or sigmoid, group_score max or sum2")
    ids, weights = (None, None) if out is None else out
    return Routing._make((_EXT or _load()).route(
        logits, top_k, _SCORES[scores], bias, groups, groups if top_groups is None else top_groups,
        _GROUP_SCORES[group_score], renormalize, scaling, ids, weights))


def expert_rows(ids, num_experts: int, token_slot=None) -> ExpertRows:
    """Sort the choices ids [T, top_k] by expert: one row per choice, stably,
    choices outside [0, num_experts) after every expert's. With token_slot
    [T], each row's adapter slot as well (what apply_linear_from_experts_
    takes, with offsets)."""
    return ExpertRows._make((_EXT or _load()).rows(ids, num_experts, token_slot))


def combine_experts(rows, positions, weights, *, residual=None, y=None):
    """y[t] = residual[t] + sum over j of weights[t, j] * rows[positions[t, j]]
    in float32, rounded once; positions outside the rows add nothing. residual
    may be y itself (an in-place sum)."""
    return (_EXT or _load()).combine(rows, positions, weights, residual, y)[0]


def quantize_mxfp4(x) -> MXFP4:
    """x [..., K] (bf16 or float32, K a multiple of 32) in MXFP4: per 32
    values a power-of-two scale from the largest of them, and the nearest
    4-bit values. A block that holds a NaN or an infinity becomes NaN."""
    _, codes, scales = (_EXT or _load()).quantize(0, x, None)
    if x.dim() != 2:
        codes = codes.view(*x.shape[:-1], codes.shape[1])
        scales = scales.view(*x.shape[:-1], scales.shape[1])
    return MXFP4(codes, scales)


def gather_quantize_mxfp4(x, row_token):
    """The rows x[row_token] (an expert-sorted batch from its tokens), as they
    are and in MXFP4: (rows, MXFP4). Indices are clamped to x's rows."""
    rows, codes, scales = (_EXT or _load()).quantize(1, x, row_token)
    return rows, MXFP4(codes, scales)


def silu_mul_quantize_mxfp4(gate_up):
    """silu(gate) * up of gate_up [rows, 2 K] (gate in the first K columns),
    in gate_up's type and in MXFP4: (rows, MXFP4)."""
    rows, codes, scales = (_EXT or _load()).quantize(2, gate_up, None)
    return rows, MXFP4(codes, scales)


def dequantize_mxfp4(q: MXFP4, dtype=None):
    """The values an MXFP4 pair stands for, in dtype (bf16 unless given)."""
    out = (_EXT or _load()).dequantize(q, dtype)[0]
    return out if q[0].dim() == 2 else out.view(*q[0].shape[:-1], out.shape[1])


def mxfp4_linear(x: MXFP4, w: MXFP4, *, dtype=None, y=None):
    """y = x @ w^T for x [rows, K] and w [N, K] in MXFP4 (w: the shards of a
    fused projection stacked along N), accumulated in float32; y is bf16
    unless dtype or y says float32. A target's LoRA delta goes onto y with
    apply_linear_."""
    return (_EXT or _load()).linear(x, w, None, dtype, y)[0]


def mxfp4_expert_linear(x: MXFP4, w: MXFP4, offsets, *, dtype=None, y=None):
    """Each row of the expert-sorted x [rows, K] against its expert's weight
    of w [experts, N, K], offsets [experts + 1] the experts' bounds; rows
    outside them become 0. The experts' LoRA goes onto y with
    apply_linear_from_experts_."""
    if offsets is None:
        raise LoraError("mxfp4_expert_linear: offsets must be [experts + 1]")
    return (_EXT or _load()).linear(x, w, offsets, dtype, y)[0]
