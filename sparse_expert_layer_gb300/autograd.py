"""Sorting tokens by expert and back inside a torch graph.

    x_sorted, plan = sort_tokens(x, topk_ids, n_experts)
    y_sorted = experts(x_sorted, plan.offsets)
    out = unsort_tokens(y_sorted, topk_w, plan)

Forward and backward are the kernels of moe_sort_tokens, moe_unsort_tokens and
their gradients (include/moe.h): sums in fp32 in slot order, the same bits on
every call.  Gradients reach x, y_sorted and topk_w; rows of dropped picks are
zero in x_sorted and in the gradient of y_sorted.  First derivatives only.
"""
from __future__ import annotations

import dataclasses

import torch
from torch.autograd.function import once_differentiable

from . import operators as ops


@dataclasses.dataclass
class SortPlan:
    """The sorted order of a batch's picks, on the device (include/moe.h)."""
    counts: torch.Tensor
    offsets: torch.Tensor
    sorted_to_expanded: torch.Tensor
    expanded_to_sorted: torch.Tensor


def _ready(t):
    """t itself where the kernels take it, else a copy (rows that are not
    contiguous or overlap, or a start that is not 16-byte aligned)."""
    fits = t.dim() == 2 and (t.shape[1] <= 1 or t.stride(1) == 1) and \
        (t.shape[0] <= 1 or t.stride(0) >= t.shape[1]) and t.data_ptr() % 16 == 0
    return t if fits else t.clone(memory_format=torch.contiguous_format)


class _Sort(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, ids, n_experts):
        T, k = ids.shape
        ids = _ready(ids).contiguous()
        i32 = dict(dtype=torch.int32, device=ids.device)
        plan = (torch.empty(n_experts, **i32), torch.empty(n_experts + 1, **i32),
                torch.empty(T * k, **i32), torch.empty(T * k, **i32))
        x_sorted = torch.empty(T * k, x.shape[1], dtype=x.dtype, device=x.device)
        ops.moe_sort_tokens(n_experts, ids, _ready(x), None, *plan, x_sorted,
                            ws=ops.sort_workspace(T, k, n_experts, x.device), zero_dropped=True)
        ctx.save_for_backward(plan[1], plan[3])
        ctx.sizes = x.shape, x.dtype, k
        ctx.mark_non_differentiable(*plan)
        return x_sorted, *plan

    @staticmethod
    @once_differentiable
    def backward(ctx, dx_sorted, *_):
        offsets, expanded_to_sorted = ctx.saved_tensors
        shape, dtype, k = ctx.sizes
        dx = torch.empty(shape, dtype=dtype, device=dx_sorted.device)
        ops.moe_sort_tokens_backward(_ready(dx_sorted).contiguous(), offsets, expanded_to_sorted, k,
                                     dx)
        return dx, None, None


class _Unsort(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y_sorted, topk_w, offsets, expanded_to_sorted, dtype):
        y, w = _ready(y_sorted).contiguous(), _ready(topk_w).contiguous()
        out = torch.empty(w.shape[0], y.shape[1], dtype=dtype, device=y.device)
        ops.moe_unsort_tokens(y, offsets, expanded_to_sorted, w, out)
        ctx.save_for_backward(y, w, offsets, expanded_to_sorted)
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        y, w, offsets, expanded_to_sorted = ctx.saved_tensors
        # frozen experts' outputs have no gradient to fill
        dy = torch.empty_like(y) if ctx.needs_input_grad[0] else None
        dw = torch.empty_like(w)
        ops.moe_unsort_tokens_backward(_ready(dout), y, offsets, expanded_to_sorted, w, dy, dw)
        return dy, dw if ctx.needs_input_grad[1] else None, None, None, None


def sort_tokens(x, topk_ids, n_experts):
    """(x_sorted [T*k, H], SortPlan) of x [T, H] (bf16, fp16 or fp32) and int32
    topk_ids [T, k]; ids outside [0, n_experts) are dropped picks.  x and topk_ids
    of other layouts are copied first."""
    if x.dtype not in (torch.bfloat16, torch.float16, torch.float32):
        raise TypeError(f"x: {x.dtype} has no gradient here")
    x_sorted, *plan = _Sort.apply(x, topk_ids, n_experts)
    return x_sorted, SortPlan(*plan)


def unsort_tokens(y_sorted, topk_w, plan, dtype=None):
    """[T, H] sums of the tokens' rows of y_sorted [T*k, H] times topk_w [T, k]
    (fp32), in `dtype` (None: y_sorted's)."""
    return _Unsort.apply(y_sorted, topk_w, plan.offsets, plan.expanded_to_sorted,
                         dtype or y_sorted.dtype)
