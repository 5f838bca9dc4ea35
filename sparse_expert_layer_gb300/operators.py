"""Bindings of the operators around the expert layer (include/moe.h).

Functions carry the C names and write into tensors that the caller gives, on
torch's current stream unless one is passed.  Shapes, types and strides are
checked here, before the pointers reach the library: a TypeError or ValueError
names the argument; what the library refuses raises MoeError.
"""
from __future__ import annotations

import ctypes

import torch

from . import MoeError, _check, _ptr, _stream, lib  # noqa: F401

DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2, torch.int8: 3,
          torch.float8_e4m3fn: 4}
_FLOATS = (torch.bfloat16, torch.float16, torch.float32)


def _tensor(t, name, dtype, shape, like=None):
    """t is a contiguous tensor of the given dtype (one, or several to choose
    from) and shape, on the device of `like` (None: the current CUDA device)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a tensor, got {type(t).__name__}")
    if t.dtype != dtype and not (isinstance(dtype, tuple) and t.dtype in dtype):
        raise TypeError(f"{name}: {t.dtype} is not {dtype}")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)} is not {shape}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: not contiguous")
    _device(t, name, like)
    return t.data_ptr()


def _rows(t, name, dtype, shape, like=None):
    """(pointer, row stride) of a matrix whose rows are contiguous."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a tensor, got {type(t).__name__}")
    if t.dtype != dtype and not (isinstance(dtype, tuple) and t.dtype in dtype):
        raise TypeError(f"{name}: {t.dtype} is not {dtype}")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)} is not {shape}")
    row, step = t.stride()
    if shape[1] > 1 and step != 1:
        raise ValueError(f"{name}: channels are not contiguous")
    if shape[0] <= 1:
        row = shape[1]
    elif row < shape[1]:
        raise ValueError(f"{name}: rows overlap (stride {row})")
    _device(t, name, like)
    return t.data_ptr(), row


def _device(t, name, like):
    if like is None:
        if not t.is_cuda or t.device.index != torch.cuda.current_device():
            raise ValueError(f"{name}: not on the current CUDA device ({t.device})")
    elif t.device != like.device:
        raise ValueError(f"{name}: on {t.device}, not {like.device}")


def _matrix_shape(t, name):
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise TypeError(f"{name}: expected a matrix")
    return tuple(t.shape)


def moe_add_rmsnorm(x, residual, gamma, eps, sum_out, y=None, q=None, q_scale=None, q_group=0,
                    stream=None):
    """r = x + residual; y = r / sqrt(mean(r^2) + eps) * gamma; int8 or e4m3 codes
    of y with a scale per row (q_group 0) or per q_group channels.

    x, residual, sum_out, y [T, H] and gamma [H] share one type (bf16, fp16,
    fp32) and may have row strides; q [T, H] is int8 or float8_e4m3fn, q_scale
    fp32 [T, groups].  residual, gamma and each output may be None; sum_out may
    be x or residual itself.
    """
    T, H = shape = _matrix_shape(x, "x")
    dt = x.dtype
    px, ldx = _rows(x, "x", _FLOATS, shape)
    pr, ldr = (None, 0) if residual is None else _rows(residual, "residual", dt, shape, x)
    pg = None if gamma is None else _tensor(gamma, "gamma", dt, (H,), x)
    ps, lds = (None, 0) if sum_out is None else _rows(sum_out, "sum_out", dt, shape, x)
    py, ldy = (None, 0) if y is None else _rows(y, "y", dt, shape, x)
    pq = psc = None
    qdt = 0
    if q is not None:
        pq = _tensor(q, "q", (torch.int8, torch.float8_e4m3fn), shape, x)
        qdt = DTYPES[q.dtype]
        groups = (T, -(-H // q_group) if q_group else 1)
        if q_scale is None or (tuple(q_scale.shape) != groups and (q_group or q_scale.shape != (T,))):
            raise ValueError(f"q_scale: expected shape {groups}")
        psc = _tensor(q_scale, "q_scale", torch.float32, tuple(q_scale.shape), x)
    _check(lib.moe_add_rmsnorm(T, H, DTYPES[dt], px, ldx, pr, ldr, pg, eps, ps, lds, py, ldy, qdt,
                               q_group, pq, psc, _stream(stream)), "moe_add_rmsnorm")


def moe_sort_workspace_size(T, k, n_experts) -> int:
    n = ctypes.c_size_t(0)
    _check(lib.moe_sort_workspace_size(T, k, n_experts, ctypes.byref(n)),
           "moe_sort_workspace_size")
    return n.value


def sort_workspace(T, k, n_experts, device="cuda"):
    """A uint8 tensor of moe_sort_workspace_size bytes, or None when that is 0."""
    n = moe_sort_workspace_size(T, k, n_experts)
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def moe_sort_tokens(n_experts, ids, x, x_scale, counts, offsets, sorted_to_expanded,
                    expanded_to_sorted, x_sorted, scale_sorted=None, ws=None, zero_dropped=False,
                    stream=None):
    """Stable order of the picks ids [T, k] by expert (dropped picks last) and the
    tokens' rows x [T, H] (and fp32 scales x_scale [T]) in it.  x and x_sorted may
    be None together: only the order is wanted."""
    T, k = _matrix_shape(ids, "ids")
    R = T * k
    i32 = torch.int32
    pi = _tensor(ids, "ids", i32, (T, k))
    pc = _tensor(counts, "counts", i32, (n_experts,), ids)
    po = _tensor(offsets, "offsets", i32, (n_experts + 1,), ids)
    p1 = _tensor(sorted_to_expanded, "sorted_to_expanded", i32, (R,), ids)
    p2 = _tensor(expanded_to_sorted, "expanded_to_sorted", i32, (R,), ids)
    H, ldx, dt, px, pxs, psc, pso = 0, 0, 0, None, None, None, None
    if (x is None) != (x_sorted is None):
        raise ValueError("x and x_sorted go together")
    if x is not None:
        H = _matrix_shape(x, "x")[1]
        px, ldx = _rows(x, "x", tuple(DTYPES), (T, H), ids)
        pxs = _tensor(x_sorted, "x_sorted", x.dtype, (R, H), ids)
        dt = DTYPES[x.dtype]
    if (x_scale is None) != (scale_sorted is None):
        raise ValueError("x_scale and scale_sorted go together")
    if x_scale is not None:
        psc = _tensor(x_scale, "x_scale", torch.float32, tuple(x_scale.shape), ids)
        if x_scale.numel() != T:
            raise ValueError(f"x_scale: expected {T} values")
        pso = _tensor(scale_sorted, "scale_sorted", torch.float32, (R,), ids)
    pw = None if ws is None else _tensor(ws, "ws", torch.uint8, tuple(ws.shape), ids)
    _check(lib.moe_sort_tokens(T, k, n_experts, H, dt, pi, px, ldx, psc, pc, po, p1, p2, pxs, pso,
                               int(zero_dropped), pw, 0 if ws is None else ws.numel(),
                               _stream(stream)), "moe_sort_tokens")


def moe_sort_tokens_backward(dx_sorted, offsets, expanded_to_sorted, k, dx, stream=None):
    """dx [T, H] = each token's kept rows of dx_sorted [T*k, H], added up."""
    T, H = _matrix_shape(dx, "dx")
    pd, ld = _rows(dx, "dx", _FLOATS, (T, H))
    pr = _tensor(dx_sorted, "dx_sorted", _FLOATS, (T * k, H), dx)
    po = _tensor(offsets, "offsets", torch.int32, tuple(offsets.shape), dx)
    p2 = _tensor(expanded_to_sorted, "expanded_to_sorted", torch.int32, (T * k,), dx)
    _check(lib.moe_sort_tokens_backward(T, k, offsets.numel() - 1, H, DTYPES[dx_sorted.dtype], pr,
                                        po, p2, DTYPES[dx.dtype], pd, ld, _stream(stream)),
           "moe_sort_tokens_backward")


def moe_unsort_tokens(y_sorted, offsets, expanded_to_sorted, topk_w, out, stream=None):
    """out [T, H] = sum over each token's kept picks of topk_w [T, k] times its
    row of y_sorted [T*k, H]."""
    T, k = _matrix_shape(topk_w, "topk_w")
    H = _matrix_shape(out, "out")[1]
    pd, ld = _rows(out, "out", _FLOATS, (T, H))
    pr = _tensor(y_sorted, "y_sorted", _FLOATS, (T * k, H), out)
    po = _tensor(offsets, "offsets", torch.int32, tuple(offsets.shape), out)
    p2 = _tensor(expanded_to_sorted, "expanded_to_sorted", torch.int32, (T * k,), out)
    pw = _tensor(topk_w, "topk_w", torch.float32, (T, k), out)
    _check(lib.moe_unsort_tokens(T, k, offsets.numel() - 1, H, DTYPES[y_sorted.dtype], pr, po, p2,
                                 pw, DTYPES[out.dtype], pd, ld, _stream(stream)),
           "moe_unsort_tokens")


def moe_unsort_tokens_backward(dout, y_sorted, offsets, expanded_to_sorted, topk_w, dy_sorted,
                               dtopk_w, zero_dropped=True, stream=None):
    """Gradients of moe_unsort_tokens: dy_sorted [T*k, H] and dtopk_w [T, k]."""
    T, k = _matrix_shape(topk_w, "topk_w")
    H = _matrix_shape(dout, "dout")[1]
    pd, ld = _rows(dout, "dout", _FLOATS, (T, H))
    py = _tensor(y_sorted, "y_sorted", _FLOATS, (T * k, H), dout)
    po = _tensor(offsets, "offsets", torch.int32, tuple(offsets.shape), dout)
    p2 = _tensor(expanded_to_sorted, "expanded_to_sorted", torch.int32, (T * k,), dout)
    pw = _tensor(topk_w, "topk_w", torch.float32, (T, k), dout)
    pg = _tensor(dy_sorted, "dy_sorted", y_sorted.dtype, (T * k, H), dout)
    pdw = _tensor(dtopk_w, "dtopk_w", torch.float32, (T, k), dout)
    _check(lib.moe_unsort_tokens_backward(T, k, offsets.numel() - 1, H, DTYPES[y_sorted.dtype],
                                          DTYPES[dout.dtype], pd, ld, py, po, p2, pw, pg, pdw,
                                          int(zero_dropped), _stream(stream)),
           "moe_unsort_tokens_backward")


def pack_w4(codes):
    """uint8 codes 0 .. 15 [..., K] (K even) as moe_w4_gemv takes them, two a byte."""
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).contiguous()


def moe_w4_gemv(x, x_scale, offsets, w, scales, zeros, out, w_up=None, scales_up=None,
                zeros_up=None, stream=None):
    """out[r] = (codes - zeros) * scales @ x[r] with the weights of row r's expert;
    with w_up, silu(first) * second.

    x [R, K] bf16, fp16 or int8 (with x_scale [R] fp32); offsets int32 [E + 1] or
    None (one expert); w, w_up uint8 [E, N, K / 2]; scales [E, N, groups] bf16,
    fp16 or fp32; zeros uint8 of their shape or None (8); out [R, N].
    """
    R, K = _matrix_shape(x, "x")
    if not isinstance(w, torch.Tensor) or w.dim() != 3:
        raise TypeError("w: expected [experts, N, K / 2]")
    E, N, _ = w.shape
    px = _tensor(x, "x", (torch.bfloat16, torch.float16, torch.int8), (R, K))
    pw = _tensor(w, "w", torch.uint8, (E, N, K // 2), x)
    if not isinstance(scales, torch.Tensor) or scales.dim() != 3:
        raise TypeError("scales: expected [experts, N, groups]")
    G = scales.shape[2]
    if G < 1 or K % G:
        raise ValueError(f"scales: {G} groups do not divide K = {K}")
    ps = _tensor(scales, "scales", _FLOATS, (E, N, G), x)
    pxs = None if x_scale is None else _tensor(x_scale, "x_scale", torch.float32,
                                               tuple(x_scale.shape), x)
    if pxs is not None and x_scale.numel() != R:
        raise ValueError(f"x_scale: expected {R} values")
    pof = None if offsets is None else _tensor(offsets, "offsets", torch.int32, (E + 1,), x)
    pz = None if zeros is None else _tensor(zeros, "zeros", torch.uint8, (E, N, G), x)
    pwu = None if w_up is None else _tensor(w_up, "w_up", torch.uint8, (E, N, K // 2), x)
    psu = None if scales_up is None else _tensor(scales_up, "scales_up", scales.dtype, (E, N, G), x)
    pzu = None if zeros_up is None else _tensor(zeros_up, "zeros_up", torch.uint8, (E, N, G), x)
    po = _tensor(out, "out", _FLOATS, (R, N), x)
    _check(lib.moe_w4_gemv(E, N, K, K // G if G > 1 else 0, R, pof, DTYPES[x.dtype], px, pxs, pw,
                           pwu, DTYPES[scales.dtype], ps, psu, pz, pzu, DTYPES[out.dtype], po,
                           _stream(stream)), "moe_w4_gemv")
