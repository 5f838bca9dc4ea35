"""Bindings of the operators around the expert layer (include/moe.h).

Functions carry the C names and write into tensors that the caller gives, on
torch's current stream unless one is passed.  Shapes, types and strides are
checked here, before the pointers reach the library: a TypeError or ValueError
names the argument; what the library refuses raises MoeError.

The functions record no graph (autograd.py has those that do).  As with torch's
own calls, what they write counts as changed for tensors that autograd has saved,
and may not require a gradient while gradients are recorded.
"""
from __future__ import annotations

import ctypes

import torch

from . import _check, lib

DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2, torch.int8: 3,
          torch.float8_e4m3fn: 4}
_FLOATS = frozenset((torch.bfloat16, torch.float16, torch.float32))
_CODES = frozenset((torch.int8, torch.float8_e4m3fn))
_ANY = frozenset(DTYPES)
_F32 = frozenset((torch.float32,))
_I32 = frozenset((torch.int32,))
_U8 = frozenset((torch.uint8,))

_W4_X = frozenset((torch.bfloat16, torch.float16, torch.int8))

_add_rmsnorm = lib.moe_add_rmsnorm
_sort_tokens = lib.moe_sort_tokens
_sort_tokens_backward = lib.moe_sort_tokens_backward
_unsort_tokens = lib.moe_unsort_tokens
_unsort_tokens_backward = lib.moe_unsort_tokens_backward
_w4_gemv = lib.moe_w4_gemv
# torch.autograd.graph.increment_version for several tensors, without its type checks
_changed = torch._C._increment_version


# A call's checks are on the path of every decoded token: the common case is a few
# attribute reads, and what is wrong with an argument is worked out only then.
def _tensor(t, name, dtypes, shape, device):
    """Address of a contiguous tensor of one of the given types and the shape, on
    CUDA device `device`."""
    try:
        if t.dtype in dtypes and t.shape == shape and t.is_contiguous() \
                and t.get_device() == device:
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(t, name, dtypes, shape, device)
    raise ValueError(f"{name}: not contiguous")


def _rows(t, name, dtypes, shape, device):
    """(address, row stride) of a matrix whose rows are contiguous."""
    try:
        if t.dtype in dtypes and t.shape == shape and t.get_device() == device:
            if t.is_contiguous():
                return t.data_ptr(), shape[1]
            row, step = t.stride()
            if shape[0] <= 1:
                row = shape[1]
            if (step == 1 or shape[1] <= 1) and row >= shape[1]:
                return t.data_ptr(), row
    except AttributeError:
        pass
    _refuse(t, name, dtypes, shape, device)
    raise ValueError(f"{name}: rows are not contiguous or overlap (strides {t.stride()})")


def _refuse_grad(name):
    if torch.is_grad_enabled():
        raise ValueError(f"{name}: requires a gradient, and the call would write it without "
                         "recording one (use torch.no_grad() where that is meant)")


def _refuse(t, name, dtypes, shape, device):
    _a_tensor(t, name)
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: {t.dtype} is not one of {sorted(map(str, dtypes))}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)} is not {tuple(shape)}")
    if t.get_device() != device:
        raise ValueError(f"{name}: on {t.device}, not on CUDA device {device}")


def _a_tensor(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a tensor, got {type(t).__name__}")


def _row_scales(t, rows, device):
    """Address of x_scale, [rows] or [rows, 1]."""
    _a_tensor(t, "x_scale")
    return _tensor(t, "x_scale", _F32, (rows, 1) if t.dim() == 2 else (rows,), device)


def _matrix(t, name, dtypes, strided=True):
    """(shape, device index, address, row stride) of the matrix that sets a call's sizes."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise TypeError(f"{name}: expected a matrix")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: {t.dtype} is not one of {sorted(map(str, dtypes))}")
    shape, device = t.shape, t.get_device()
    if t.is_contiguous():
        return shape, device, t.data_ptr(), shape[1]
    if not strided:
        raise ValueError(f"{name}: not contiguous")
    return shape, device, *_rows(t, name, dtypes, shape, device)


def _stream(stream, device):
    """The handle of the stream to launch on (None: the current one)."""
    if device < 0 or device != torch._C._cuda_getDevice():
        raise ValueError("the tensors are not on the current CUDA device")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device)
    return stream if isinstance(stream, int) else stream.cuda_stream


def moe_add_rmsnorm(x, residual, gamma, eps, sum_out, y=None, q=None, q_scale=None, q_group=0,
                    stream=None):
    """r = x + residual; y = r / sqrt(mean(r^2) + eps) * gamma; int8 or e4m3 codes
    of y with a scale per row (q_group 0) or per q_group channels.

    x, residual, sum_out, y [T, H] and gamma [H] share one type (bf16, fp16,
    fp32) and may have row strides; q [T, H] is int8 or float8_e4m3fn, q_scale
    fp32 [T, groups] ([T, 1] for q_group 0).  residual, gamma and each output may be None; sum_out may
    be x or residual itself.
    """
    shape, dev, px, ldx = _matrix(x, "x", _FLOATS)
    T, H = shape
    same = (x.dtype,)
    pr = pg = ps = py = pq = psc = None
    ldr = lds = ldy = qdt = 0
    written = []
    if residual is not None:
        pr, ldr = _rows(residual, "residual", same, shape, dev)
    if gamma is not None:
        pg = _tensor(gamma, "gamma", same, (H,), dev)
    if sum_out is not None:
        ps, lds = _rows(sum_out, "sum_out", same, shape, dev)
        if sum_out.requires_grad:
            _refuse_grad("sum_out")
        written.append(sum_out)
    if y is not None:
        py, ldy = _rows(y, "y", same, shape, dev)
        if y.requires_grad:
            _refuse_grad("y")
        written.append(y)
    if q is not None:
        pq = _tensor(q, "q", _CODES, shape, dev)
        qdt = DTYPES[q.dtype]
        psc = _tensor(q_scale, "q_scale", _F32, (T, -(-H // q_group) if q_group else 1), dev)
        if q.requires_grad or q_scale.requires_grad:
            _refuse_grad("q_scale" if q_scale.requires_grad else "q")
        written += (q, q_scale)
    st = _add_rmsnorm(T, H, DTYPES[x.dtype], px, ldx, pr, ldr, pg, eps, ps, lds, py, ldy, qdt,
                      q_group, pq, psc, _stream(stream, dev))
    if st:
        _check(st, "moe_add_rmsnorm")
    _changed(written)


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
    (T, k), dev, pi, _ = _matrix(ids, "ids", _I32, strided=False)
    R = T * k
    pc = _tensor(counts, "counts", _I32, (n_experts,), dev)
    po = _tensor(offsets, "offsets", _I32, (n_experts + 1,), dev)
    p1 = _tensor(sorted_to_expanded, "sorted_to_expanded", _I32, (R,), dev)
    p2 = _tensor(expanded_to_sorted, "expanded_to_sorted", _I32, (R,), dev)
    written = [counts, offsets, sorted_to_expanded, expanded_to_sorted]
    H = ldx = dt = nws = 0
    px = pxs = psc = pso = pw = None
    if x is not None:
        try:
            if x.dim() != 2:
                raise ValueError("x: expected a matrix")
        except AttributeError:
            _a_tensor(x, "x")
            raise
        H = x.shape[1]
        px, ldx = _rows(x, "x", _ANY, (T, H), dev)
        pxs = _tensor(x_sorted, "x_sorted", (x.dtype,), (R, H), dev)
        if x_sorted.requires_grad:
            _refuse_grad("x_sorted")
        written.append(x_sorted)
        dt = DTYPES[x.dtype]
    elif x_sorted is not None:
        raise ValueError("x_sorted: given without x")
    if x_scale is not None:
        psc = _row_scales(x_scale, T, dev)
        pso = _tensor(scale_sorted, "scale_sorted", _F32, (R,), dev)
        if scale_sorted.requires_grad:
            _refuse_grad("scale_sorted")
        written.append(scale_sorted)
    elif scale_sorted is not None:
        raise ValueError("scale_sorted: given without x_scale")
    if ws is not None:
        _a_tensor(ws, "ws")
        nws = ws.numel()
        pw = _tensor(ws, "ws", _U8, (nws,), dev)
    st = _sort_tokens(T, k, n_experts, H, dt, pi, px, ldx, psc, pc, po, p1, p2, pxs, pso,
                      1 if zero_dropped else 0, pw, nws, _stream(stream, dev))
    if st:
        _check(st, "moe_sort_tokens")
    _changed(written)


def _picks(topk_w):
    try:
        return topk_w.shape[1]
    except (AttributeError, IndexError):
        _matrix(topk_w, "topk_w", _F32)  # says what is wrong
        raise


def _plan(offsets, expanded_to_sorted, R, dev):
    """(experts, addresses) of the plan that moe_sort_tokens wrote."""
    try:
        E = offsets.numel() - 1
    except AttributeError:
        _a_tensor(offsets, "offsets")
        raise
    return E, _tensor(offsets, "offsets", _I32, (E + 1,), dev), \
        _tensor(expanded_to_sorted, "expanded_to_sorted", _I32, (R,), dev)


def moe_sort_tokens_backward(dx_sorted, offsets, expanded_to_sorted, k, dx, stream=None):
    """dx [T, H] = each token's kept rows of dx_sorted [T*k, H], added up."""
    (T, H), dev, pd, ld = _matrix(dx, "dx", _FLOATS)
    if dx.requires_grad:
        _refuse_grad("dx")
    pr = _tensor(dx_sorted, "dx_sorted", _FLOATS, (T * k, H), dev)
    E, po, p2 = _plan(offsets, expanded_to_sorted, T * k, dev)
    st = _sort_tokens_backward(T, k, E, H, DTYPES[dx_sorted.dtype], pr, po, p2, DTYPES[dx.dtype],
                               pd, ld, _stream(stream, dev))
    if st:
        _check(st, "moe_sort_tokens_backward")
    _changed((dx,))


def moe_unsort_tokens(y_sorted, offsets, expanded_to_sorted, topk_w, out, stream=None):
    """out [T, H] = sum over each token's kept picks of topk_w [T, k] times its
    row of y_sorted [T*k, H]."""
    (T, H), dev, pd, ld = _matrix(out, "out", _FLOATS)
    k = _picks(topk_w)
    if out.requires_grad:
        _refuse_grad("out")
    pr = _tensor(y_sorted, "y_sorted", _FLOATS, (T * k, H), dev)
    E, po, p2 = _plan(offsets, expanded_to_sorted, T * k, dev)
    pw = _tensor(topk_w, "topk_w", _F32, (T, k), dev)
    st = _unsort_tokens(T, k, E, H, DTYPES[y_sorted.dtype], pr, po, p2, pw, DTYPES[out.dtype], pd,
                        ld, _stream(stream, dev))
    if st:
        _check(st, "moe_unsort_tokens")
    _changed((out,))


def moe_unsort_tokens_backward(dout, y_sorted, offsets, expanded_to_sorted, topk_w, dy_sorted,
                               dtopk_w, zero_dropped=True, stream=None):
    """Gradients of moe_unsort_tokens: dy_sorted [T*k, H] (None: not wanted) and
    dtopk_w [T, k]."""
    (T, H), dev, pd, ld = _matrix(dout, "dout", _FLOATS)
    k = _picks(topk_w)
    py = _tensor(y_sorted, "y_sorted", _FLOATS, (T * k, H), dev)
    E, po, p2 = _plan(offsets, expanded_to_sorted, T * k, dev)
    pw = _tensor(topk_w, "topk_w", _F32, (T, k), dev)
    pdw = _tensor(dtopk_w, "dtopk_w", _F32, (T, k), dev)
    if dtopk_w.requires_grad:
        _refuse_grad("dtopk_w")
    written, pg = [dtopk_w], None
    if dy_sorted is not None:
        pg = _tensor(dy_sorted, "dy_sorted", (y_sorted.dtype,), (T * k, H), dev)
        if dy_sorted.requires_grad:
            _refuse_grad("dy_sorted")
        written.append(dy_sorted)
    st = _unsort_tokens_backward(T, k, E, H, DTYPES[y_sorted.dtype], DTYPES[dout.dtype], pd, ld, py,
                                 po, p2, pw, pg, pdw, 1 if zero_dropped else 0,
                                 _stream(stream, dev))
    if st:
        _check(st, "moe_unsort_tokens_backward")
    _changed(written)


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
    (R, K), dev, px, _ = _matrix(x, "x", _W4_X, strided=False)
    if not isinstance(w, torch.Tensor) or w.dim() != 3:
        raise TypeError("w: expected [experts, N, K / 2]")
    E, N, _ = w.shape
    if not isinstance(scales, torch.Tensor) or scales.dim() != 3:
        raise TypeError("scales: expected [experts, N, groups]")
    G = scales.shape[2]
    if G < 1 or K % G:
        raise ValueError(f"scales: {G} groups do not divide K = {K}")
    wshape, gshape = (E, N, K // 2), (E, N, G)
    pw = _tensor(w, "w", _U8, wshape, dev)
    ps = _tensor(scales, "scales", _FLOATS, gshape, dev)
    pxs = pof = pz = pwu = psu = pzu = None
    if x_scale is not None:
        pxs = _row_scales(x_scale, R, dev)
    if offsets is not None:
        pof = _tensor(offsets, "offsets", _I32, (E + 1,), dev)
    if zeros is not None:
        pz = _tensor(zeros, "zeros", _U8, gshape, dev)
    if w_up is not None:
        pwu = _tensor(w_up, "w_up", _U8, wshape, dev)
    if scales_up is not None:
        psu = _tensor(scales_up, "scales_up", (scales.dtype,), gshape, dev)
    if zeros_up is not None:
        pzu = _tensor(zeros_up, "zeros_up", _U8, gshape, dev)
    po = _tensor(out, "out", _FLOATS, (R, N), dev)
    if out.requires_grad:
        _refuse_grad("out")
    st = _w4_gemv(E, N, K, K // G if G > 1 else 0, R, pof, DTYPES[x.dtype], px, pxs, pw, pwu,
                  DTYPES[scales.dtype], ps, psu, pz, pzu, DTYPES[out.dtype], po,
                  _stream(stream, dev))
    if st:
        _check(st, "moe_w4_gemv")
    _changed((out,))
