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
before it).  No call waits for the GPU except ``expert_weight_quant_matmul``
without ``bounds``.
"""
from __future__ import annotations

from typing import NamedTuple, Optional, Sequence

import torch

from . import _both_phases, _desc_bytes, _placed, _same_device, lib, weight_quant_matmul


class TokenOrder(NamedTuple):
    """The slots sorted by group (expert or adapter); int32 tensors."""
    offsets: object   # (groups + 1): group g has the sorted rows offsets[g] .. offsets[g + 1] - 1
    source: object    # (slots): the slot of every sorted row; behind offsets[groups] the slots of no group
    position: object  # shape of the ids: the sorted row of every slot, -1 for a slot of no group


def sort_tokens(expert_ids, num_experts: int, stream=None) -> TokenOrder:
    """The stable order of the slots by expert: expert_ids (T), (T, K) or (b, s, K), int32 or int64; an id outside
    [0, num_experts) belongs to no expert (a dropped slot, or an expert of another rank)."""
    device = _same_device(expert_ids)
    where = _placed(device, stream)
    if where is not None:
        with where:
            return sort_tokens(expert_ids, num_experts)
    if not expert_ids.is_contiguous():
        raise ValueError("expert_ids must be contiguous")
    offsets = expert_ids.new_empty(max(int(num_experts), 0) + 1, dtype=torch.int32)
    source = expert_ids.new_empty(expert_ids.numel(), dtype=torch.int32)
    position = torch.empty_like(expert_ids, dtype=torch.int32)
    L = lib()
    _both_phases(L.route_sort_get_workspace_size, L.route_run, device, _desc_bytes(expert_ids), int(num_experts),
                 _desc_bytes(offsets), _desc_bytes(source), _desc_bytes(position))
    return TokenOrder(offsets, source, position)


def dispatch_tokens(x, order: TokenOrder, out=None, stream=None):
    """out[position[t, j]] = x[t] for every slot of an expert; x (T, hidden) or (b, s, hidden).  ``out``: (rows,
    hidden) of x's dtype, one row per slot unless given; rows of no slot keep what they hold (in an ``out`` made
    here that is uninitialised memory, behind order.offsets[-1])."""
    device = _same_device(x, order.position, out)
    where = _placed(device, stream)
    if where is not None:
        with where:
            return dispatch_tokens(x, order, out)
    if out is None:
        out = x.new_empty((order.position.numel(), x.shape[-1]))
    L = lib()
    _both_phases(L.route_dispatch_get_workspace_size, L.route_run, device, _desc_bytes(x),
                 _desc_bytes(order.position), _desc_bytes(out))
    return out


def combine_tokens(x_sorted, order: TokenOrder, weights=None, x3=None, out=None, stream=None):
    """out[t] = x3[t] + sum_j weights[t, j] * x_sorted[position[t, j]], in 32 bits, rounded once.  ``weights``:
    shape of position, float16, bfloat16 or float32; None: all one, which is also the gradient of
    ``dispatch_tokens``.  ``out``: (T, hidden) unless x3 or ``out`` says (b, s, hidden)."""
    device = _same_device(x_sorted, order.position, weights, x3, out)
    where = _placed(device, stream)
    if where is not None:
        with where:
            return combine_tokens(x_sorted, order, weights, x3, out)
    if out is None:
        if x3 is not None:
            out = torch.empty_like(x3)
        else:
            p = order.position.shape
            tokens = p if len(p) == 1 else p[:-1]
            out = x_sorted.new_empty((*tokens, x_sorted.shape[-1]))
    L = lib()
    _both_phases(L.route_combine_get_workspace_size, L.route_run, device, _desc_bytes(x_sorted),
                 _desc_bytes(order.position), _desc_bytes(weights), _desc_bytes(x3), _desc_bytes(out))
    return out


def combine_tokens_grad(grad, x_sorted, order: TokenOrder, weights, out=None, stream=None):
    """The gradient of ``combine_tokens`` for x_sorted and weights, given ``grad`` of its result:
    (grad_sorted, grad_weights).  Rows of no slot keep what ``out`` (grad_sorted's tensor, made here unless given)
    holds; grad_weights of a slot of no expert is 0."""
    device = _same_device(grad, x_sorted, order.position, weights, out)
    where = _placed(device, stream)
    if where is not None:
        with where:
            return combine_tokens_grad(grad, x_sorted, order, weights, out)
    if out is None:
        out = torch.empty_like(x_sorted)
    grad_weights = torch.empty_like(weights)
    L = lib()
    _both_phases(L.route_combine_grad_get_workspace_size, L.route_run, device, _desc_bytes(grad),
                 _desc_bytes(x_sorted), _desc_bytes(order.position), _desc_bytes(weights), _desc_bytes(out),
                 _desc_bytes(grad_weights))
    return out, grad_weights


def expert_weight_quant_matmul(x_sorted, order: TokenOrder, x2_descs: Sequence, antiquant_scales: Sequence,
                               antiquant_offsets: Optional[Sequence] = None, biases: Optional[Sequence] = None,
                               antiquant_group_size: int = 0, out=None, bounds: Optional[Sequence[int]] = None,
                               stream=None):
    """out[rows of e] = the anti-quant GEMM of expert e's rows of x_sorted with its weight, for every expert that
    has rows.  ``bounds``: order.offsets on the host (None: read here, which waits for the stream).  Rows behind
    the last expert keep what ``out`` holds."""
    device = _same_device(x_sorted, out)
    where = _placed(device, stream)
    if where is not None:
        with where:
            return expert_weight_quant_matmul(x_sorted, order, x2_descs, antiquant_scales, antiquant_offsets, biases,
                                              antiquant_group_size, out, bounds)
    if bounds is None:
        bounds = order.offsets.tolist()
    if len(bounds) != len(x2_descs) + 1:
        raise ValueError(f"{len(x2_descs)} weights for {len(bounds) - 1} experts")
    if out is None:
        out = x_sorted.new_empty((x_sorted.shape[0], x2_descs[0].shape[1]))
    for e, desc in enumerate(x2_descs):
        lo, hi = bounds[e], bounds[e + 1]
        if lo < hi:
            weight_quant_matmul(x_sorted[lo:hi], desc, antiquant_scales[e],
                                None if antiquant_offsets is None else antiquant_offsets[e],
                                None if biases is None else biases[e],
                                antiquant_group_size=antiquant_group_size, out=out[lo:hi])
    return out
