"""Low-rank adapters of many requests beside a shared quantised projection, and their gradients.

Every row of a batch has one adapter or none.  ``adapter_order`` sorts the rows
by adapter once per batch; every projection of every layer then reads that
order: ``lora_add`` adds the adapters' part to a projection's output (in place
if asked), ``lora_weight_quant_matmul`` runs the quantised projection and that,
and ``lora_grad`` gives the gradients for the input and the adapters (the
projection's weight is frozen).

Every call works on the tensors' device and on its current stream, or on
``stream`` (a torch.cuda.Stream or a raw handle; the caller orders the inputs
before it and keeps them until it has run), and does not wait for the GPU.
"""
from __future__ import annotations

import torch

from . import _on_stream, _same_device, _share_memory, binding, weight_quant_matmul
from .routing import TokenOrder, sort_tokens


def adapter_order(adapter_ids, num_adapters: int, stream=None) -> TokenOrder:
    """The rows in the order of their adapters: adapter_ids (m), one index per row, int32 or int64; an index outside
    [0, num_adapters) is a row without adapter.  For x1 of (b, s, k) the rows are counted through."""
    if stream is not None:
        with _on_stream(stream, _same_device(adapter_ids)):  # where a copy that reshape makes belongs too
            return adapter_order(adapter_ids, num_adapters)
    return sort_tokens(adapter_ids.reshape(-1), num_adapters)


def lora_add(x1, lora_a, lora_b, order: TokenOrder, scale=None, y=None, out=None, stream=None):
    """out[r] = y[r] + scale[a] * (x1[r] @ lora_a[a].T) @ lora_b[a].T, a the adapter of row r; a row without adapter
    gets y, or zeros.  x1 (m, k) or (b, s, k); lora_a (adapters, rank, k); lora_b (adapters, n, rank); scale
    (adapters) float32; ``out`` may be ``y``, and ``x1`` where k = n, and shares no other memory with them."""
    if stream is not None:
        with _on_stream(stream, _same_device(x1, lora_a, lora_b, order.offsets, order.source, scale, y, out)):
            return lora_add(x1, lora_a, lora_b, order, scale, y, out)
    return binding().lora_add(x1, lora_a, lora_b, scale, order.offsets, order.source, y, out)


def lora_weight_quant_matmul(x1, x2_desc, antiquant_scale, lora_a, lora_b, order: TokenOrder, lora_scale=None,
                             antiquant_offset=None, bias=None, x3=None, antiquant_group_size: int = 0, out=None,
                             stream=None):
    """The anti-quant projection of x1 with the rows' adapters added in place:
    out = x1 @ ((x2 + antiquant_offset) * antiquant_scale) + bias + x3 + the adapters' part.  The projection is
    rounded to the output type before the adapters' part is added, and the sum once more.  ``out`` may not share
    memory with x1, which the adapters read behind the projection."""
    device = _same_device(x1, antiquant_scale, antiquant_offset, bias, x3, out, lora_a, lora_b, order.offsets,
                          order.source, lora_scale)
    if stream is not None or device != torch.cuda.current_device():
        with torch.cuda.device(device) if stream is None else _on_stream(stream, device):
            return lora_weight_quant_matmul(x1, x2_desc, antiquant_scale, lora_a, lora_b, order, lora_scale,
                                            antiquant_offset, bias, x3, antiquant_group_size, out)
    if out is not None:
        # the adapters' arguments are refused before the projection has written the caller's tensor
        if _share_memory(out, x1):
            raise ValueError("out shares memory with x1")
        binding().check_lora_add(x1, lora_a, lora_b, lora_scale, order.offsets, order.source, out, out)
    out = weight_quant_matmul(x1, x2_desc, antiquant_scale, antiquant_offset, bias, x3, antiquant_group_size, out)
    return lora_add(x1, lora_a, lora_b, order, lora_scale, y=out, out=out)


def lora_grad(grad, x1, lora_a, lora_b, order: TokenOrder, scale=None, grad_x=None, need_grad_x: bool = True,
              in_place: bool = False, stream=None):
    """The gradients of ``lora_add`` given ``grad`` of its result (y's is ``grad`` itself): (for x1, lora_a, lora_b).
    ``grad_x`` (m, k): what else x1's gradient has, the projection's own part, added in 32 bits before the one
    rounding; with ``in_place`` the sum goes into that tensor (which may be ``grad`` itself where k = n, or ``x1``).
    ``need_grad_x`` False: None in x1's place.  At most 2^24 rows."""
    if stream is not None:
        with _on_stream(stream, _same_device(grad, x1, lora_a, lora_b, order.offsets, order.source, scale, grad_x)):
            return lora_grad(grad, x1, lora_a, lora_b, order, scale, grad_x, need_grad_x, in_place)
    if grad_x is None and in_place:
        raise ValueError("in_place needs a grad_x to add to")
    if grad_x is not None and not need_grad_x:
        raise ValueError("a grad_x is given, but need_grad_x is False")
    return binding().lora_grad(grad, x1, lora_a, lora_b, scale, order.offsets, order.source, grad_x, need_grad_x,
                               in_place)
