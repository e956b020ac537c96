"""Tokens sorted by expert and back, around the experts' quantised products.

``sort_tokens`` gives the stable order of the slots -- a slot is one (token,
choice) pair -- by expert, ``dispatch_tokens`` copies the tokens into it,
``expert_weight_quant_matmul`` multiplies every expert's rows with its
quantised weight, and ``combine_tokens`` sums the experts' rows of every token
with the router's weights.  The gradients: of ``dispatch_tokens``
``combine_tokens`` without weights, of ``combine_tokens``
``combine_tokens_grad``.  The same order by adapter is what the low-rank
adapters of ``lora`` read.

Every call works on the tensors' device and on its current stream, or on
``stream`` (a torch.cuda.Stream or a raw handle; the caller orders the inputs
before it and keeps them until it has run).  No call waits for the GPU except
``expert_weight_quant_matmul`` without ``bounds``.
"""
from __future__ import annotations

from typing import NamedTuple, Optional, Sequence

import torch

from . import _on_stream, _same_device, _share_memory, binding, weight_quant_matmul


class TokenOrder(NamedTuple):
    """The slots sorted by group (expert or adapter); int32 tensors."""
    offsets: object   # (groups + 1): group g has the sorted rows offsets[g] .. offsets[g + 1] - 1
    source: object    # (slots): the slot of every sorted row; behind offsets[groups] the slots of no group
    position: object  # shape of the ids: the sorted row of every slot, -1 for a slot of no group


def sort_tokens(expert_ids, num_experts: int, stream=None) -> TokenOrder:
    """The stable order of the slots by expert: expert_ids (T), (T, K) or (b, s, K), int32 or int64; an id outside
    [0, num_experts) belongs to no expert (a dropped slot, or an expert of another rank)."""
    if stream is not None:
        with _on_stream(stream, _same_device(expert_ids)):
            return sort_tokens(expert_ids, num_experts)
    return TokenOrder(*binding().sort_tokens(expert_ids, num_experts))


def dispatch_tokens(x, order: TokenOrder, out=None, stream=None):
    """out[position[t, j]] = x[t] for every slot of an expert; x (T, hidden) or (b, s, hidden).  ``out``: (rows,
    hidden) of x's dtype, one row per slot unless given; rows of no slot keep what they hold (in an ``out`` made
    here that is uninitialised memory, behind order.offsets[-1])."""
    if stream is not None:
        with _on_stream(stream, _same_device(x, order.position, out)):
            return dispatch_tokens(x, order, out)
    return binding().dispatch_tokens(x, order.position, out)


def combine_tokens(x_sorted, order: TokenOrder, weights=None, x3=None, out=None, stream=None):
    """out[t] = x3[t] + sum_j weights[t, j] * x_sorted[position[t, j]], in 32 bits, rounded once.  ``weights``:
    shape of position, float16, bfloat16 or float32; None: all one, which is also the gradient of
    ``dispatch_tokens``.  ``out``: (T, hidden) unless x3 or ``out`` says (b, s, hidden); it may be x3 itself."""
    if stream is not None:
        with _on_stream(stream, _same_device(x_sorted, order.position, weights, x3, out)):
            return combine_tokens(x_sorted, order, weights, x3, out)
    return binding().combine_tokens(x_sorted, order.position, weights, x3, out)


def combine_tokens_grad(grad, x_sorted, order: TokenOrder, weights, out=None, stream=None):
    """The gradient of ``combine_tokens`` for x_sorted and weights, given ``grad`` of its result:
    (grad_sorted, grad_weights).  Rows of no slot keep what ``out`` (grad_sorted's tensor) holds (in an ``out`` made
    here that is uninitialised memory); it may be x_sorted itself.  grad_weights of a slot of no expert is 0."""
    if stream is not None:
        with _on_stream(stream, _same_device(grad, x_sorted, order.position, weights, out)):
            return combine_tokens_grad(grad, x_sorted, order, weights, out)
    return binding().combine_tokens_grad(grad, x_sorted, order.position, weights, out)


def expert_weight_quant_matmul(x_sorted, order: TokenOrder, x2_descs: Sequence, antiquant_scales: Sequence,
                               antiquant_offsets: Optional[Sequence] = None, biases: Optional[Sequence] = None,
                               antiquant_group_size: int = 0, out=None, bounds: Optional[Sequence[int]] = None,
                               stream=None):
    """out[rows of e] = the anti-quant GEMM of expert e's rows of x_sorted with its weight, for every expert that
    has rows.  The lists have one entry per expert (a bias, offset or, for weights that are not quantised, scale may
    be None).  ``bounds``: order.offsets on the host (None: read here, which waits for the stream).  An x_sorted of
    fewer rows than slots has no rows for what lies behind.  Rows behind the last expert keep what ``out`` holds;
    ``out`` may not share memory with x_sorted."""
    device = _same_device(x_sorted, out)
    if stream is not None or device != torch.cuda.current_device():
        with torch.cuda.device(device) if stream is None else _on_stream(stream, device):
            return expert_weight_quant_matmul(x_sorted, order, x2_descs, antiquant_scales, antiquant_offsets, biases,
                                              antiquant_group_size, out, bounds)
    if len(x2_descs) == 0:
        raise ValueError("no experts")
    for name, entries in (("antiquant_scales", antiquant_scales), ("antiquant_offsets", antiquant_offsets),
                          ("biases", biases)):
        if entries is not None and len(entries) != len(x2_descs):
            raise ValueError(f"{len(entries)} {name} for {len(x2_descs)} weights")
    if x_sorted.dim() != 2:
        raise ValueError(f"x_sorted must be 2-D (rows, hidden), got {x_sorted.dim()}-D")
    if bounds is None:
        bounds = order.offsets.tolist()
    if len(bounds) != len(x2_descs) + 1:
        raise ValueError(f"{len(x2_descs)} weights for {len(bounds) - 1} experts")
    if bounds[0] < 0 or any(lo > hi for lo, hi in zip(bounds, bounds[1:])):
        raise ValueError("bounds must ascend from 0 or more")
    bounds = [min(b, x_sorted.shape[0]) for b in bounds]
    if out is not None:
        if out.dim() != 2 or out.shape[0] < bounds[-1]:
            raise ValueError(f"out must be 2-D with {bounds[-1]} rows or more, got {tuple(out.shape)}")
        if _share_memory(out, x_sorted):
            raise ValueError("out shares memory with x_sorted")
    if out is None:
        out = x_sorted.new_empty((x_sorted.shape[0], x2_descs[0].shape[1]))
    for e, desc in enumerate(x2_descs):
        lo, hi = bounds[e], bounds[e + 1]
        if lo < hi:
            weight_quant_matmul(x_sorted[lo:hi], desc, None if antiquant_scales is None else antiquant_scales[e],
                                None if antiquant_offsets is None else antiquant_offsets[e],
                                None if biases is None else biases[e],
                                antiquant_group_size=antiquant_group_size, out=out[lo:hi])
    return out
