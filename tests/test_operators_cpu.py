"""The operators around the layer refuse bad arguments on the host, before any
launch: through the C ABI with addresses that are never read, and through the
Python binding's checks with CPU tensors."""
import ctypes

import pytest
import torch

FAKE = 1 << 40  # never dereferenced
BF16, FP16, FP32, INT8, E4M3 = range(5)
INVALID, UNSUPPORTED, ALIGNMENT, WS = 1, 2, 3, 4


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__

    __graft_entry__._builder().build()
    import sparse_expert_layer_gb300 as m

    return m


def norm(moe, **kw):
    a = dict(T=4, H=64, dtype=BF16, x=FAKE, ldx=64, res=FAKE, ldr=64, gamma=FAKE, eps=1e-6,
             sum=FAKE, lds=64, y=FAKE, ldy=64, q_dtype=INT8, q_group=0, q=FAKE, scale=FAKE)
    a.update(kw)
    return moe.lib.moe_add_rmsnorm(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(dtype=INT8), INVALID),
    (dict(dtype=-1), INVALID), (dict(eps=-1e-6), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(eps=float("inf")), INVALID), (dict(ldx=63), INVALID), (dict(ldr=63), INVALID),
    (dict(lds=63), INVALID), (dict(ldy=63), INVALID), (dict(q_dtype=BF16), INVALID),
    (dict(q_group=48), INVALID), (dict(q_group=-32), INVALID), (dict(q_group=512), INVALID),
    (dict(sum=None, y=None, q=None), INVALID), (dict(x=None), INVALID),
    (dict(scale=None), INVALID), (dict(H=32769, ldx=40000, ldr=40000, lds=40000, ldy=40000),
                                  UNSUPPORTED),
    (dict(x=FAKE + 2), ALIGNMENT), (dict(res=FAKE + 8), ALIGNMENT),
    (dict(gamma=FAKE + 4), ALIGNMENT), (dict(q=FAKE + 1), ALIGNMENT),
    (dict(scale=FAKE + 4), ALIGNMENT), (dict(y=FAKE + 2), ALIGNMENT),
])
def test_norm_refusals(moe, kw, status):
    assert norm(moe, **kw) == status


def test_norm_without_rows_is_a_no_op(moe):
    assert norm(moe, T=0, x=None, res=None, gamma=None) == 0


def sort(moe, **kw):
    a = dict(T=4, k=2, E=8, H=64, dtype=BF16, ids=FAKE, x=FAKE, ldx=64, x_scale=None, counts=FAKE,
             offsets=FAKE, s2e=FAKE, e2s=FAKE, xs=FAKE, ss=None, zero=0, ws=None, ws_bytes=0)
    a.update(kw)
    return moe.lib.moe_sort_tokens(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INVALID), (dict(k=0), INVALID), (dict(k=33), UNSUPPORTED), (dict(E=0), INVALID),
    (dict(E=4097), UNSUPPORTED), (dict(T=1 << 30, k=2), UNSUPPORTED), (dict(H=0), INVALID),
    (dict(dtype=7), INVALID), (dict(ldx=63), INVALID), (dict(ids=None), INVALID),
    (dict(x=None), INVALID), (dict(counts=None), INVALID), (dict(offsets=None), INVALID),
    (dict(s2e=None), INVALID), (dict(e2s=None), INVALID), (dict(zero=2), INVALID),
    (dict(ss=FAKE), INVALID), (dict(xs=None, ss=FAKE, x_scale=FAKE), INVALID),
    (dict(x=FAKE + 2), ALIGNMENT), (dict(xs=FAKE + 8), ALIGNMENT), (dict(ids=FAKE + 4), ALIGNMENT),
    (dict(T=8192, k=8), INVALID),                                   # needs a workspace
    (dict(T=8192, k=8, ws=FAKE + 16, ws_bytes=1 << 30), ALIGNMENT),
    (dict(T=8192, k=8, ws=FAKE, ws_bytes=64), WS),
])
def test_sort_refusals(moe, kw, status):
    assert sort(moe, **kw) == status


def test_sort_workspace_size(moe):
    assert moe.moe_sort_workspace_size(16, 2, 8) == 0
    a, b = (moe.moe_sort_workspace_size(T, 8, 256) for T in (8192, 16384))
    assert 0 < a < b
    n = ctypes.c_size_t(0)
    assert moe.lib.moe_sort_workspace_size(16, 0, 8, ctypes.byref(n)) == INVALID
    assert moe.lib.moe_sort_workspace_size(16, 2, 8, None) == INVALID


def back(moe, **kw):
    a = dict(T=4, k=2, E=8, H=64, dtype=BF16, rows=FAKE, offsets=FAKE, e2s=FAKE, w=FAKE,
             out_dtype=FP32, out=FAKE, ldo=64)
    a.update(kw)
    return moe.lib.moe_unsort_tokens(*a.values(), None)


def grad(moe, **kw):
    a = dict(T=4, k=2, E=8, H=64, dtype=BF16, out_dtype=FP32, dout=FAKE, ldd=64, rows=FAKE,
             offsets=FAKE, e2s=FAKE, w=FAKE, drows=FAKE, dw=FAKE, zero=1)
    a.update(kw)
    return moe.lib.moe_unsort_tokens_backward(*a.values(), None)


COMMON = [(dict(T=-1), INVALID), (dict(k=0), INVALID), (dict(k=33), UNSUPPORTED),
          (dict(E=4097), UNSUPPORTED), (dict(H=0), INVALID), (dict(dtype=INT8), INVALID),
          (dict(out_dtype=E4M3), INVALID), (dict(rows=None), INVALID),
          (dict(offsets=None), INVALID), (dict(e2s=None), INVALID), (dict(w=None), INVALID),
          (dict(rows=FAKE + 2), ALIGNMENT), (dict(w=FAKE + 4), ALIGNMENT)]


@pytest.mark.parametrize("kw,status", COMMON + [(dict(ldo=63), INVALID), (dict(out=None), INVALID),
                                                (dict(out=FAKE + 8), ALIGNMENT)])
def test_unsort_refusals(moe, kw, status):
    assert back(moe, **kw) == status


@pytest.mark.parametrize("kw,status", COMMON + [(dict(ldd=63), INVALID), (dict(dout=None), INVALID),
                                                (dict(dw=None), INVALID), (dict(zero=-1), INVALID),
                                                (dict(drows=FAKE + 8), ALIGNMENT)])
def test_unsort_backward_refusals(moe, kw, status):
    assert grad(moe, **kw) == status


def w4(moe, **kw):
    a = dict(E=2, N=64, K=128, group=32, R=4, offsets=FAKE, x_dtype=BF16, x=FAKE, x_scale=None,
             w=FAKE, w_up=None, scale_dtype=BF16, scales=FAKE, scales_up=None, zeros=None,
             zeros_up=None, out_dtype=BF16, out=FAKE)
    a.update(kw)
    return moe.lib.moe_w4_gemv(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(E=0), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(K=48), INVALID),
    (dict(R=-1), INVALID), (dict(group=16), INVALID), (dict(group=256), INVALID),
    (dict(group=128, K=160), INVALID), (dict(x_dtype=FP32), INVALID), (dict(x_dtype=E4M3), INVALID),
    (dict(scale_dtype=INT8), INVALID), (dict(out_dtype=INT8), INVALID),
    (dict(offsets=None), INVALID), (dict(w_up=FAKE), INVALID), (dict(scales_up=FAKE), INVALID),
    (dict(zeros_up=FAKE), INVALID), (dict(w_up=FAKE, scales_up=FAKE, zeros=FAKE), INVALID),
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(scales=None), INVALID),
    (dict(out=None), INVALID), (dict(x_scale=FAKE), INVALID), (dict(x_dtype=INT8), INVALID),
    (dict(E=4097), UNSUPPORTED), (dict(N=1 << 23), UNSUPPORTED), (dict(w=FAKE + 8), ALIGNMENT),
    (dict(x=FAKE + 2), ALIGNMENT), (dict(zeros=FAKE + 1), ALIGNMENT), (dict(out=FAKE + 4), ALIGNMENT),
])
def test_w4_refusals(moe, kw, status):
    assert w4(moe, **kw) == status


def test_w4_without_rows_is_a_no_op(moe):
    assert w4(moe, R=0, x=None, w=None, scales=None, out=None) == 0


def test_pack_w4(moe):
    codes = torch.randint(0, 16, (2, 3, 64), dtype=torch.uint8)
    packed = moe.pack_w4(codes)
    assert packed.shape == (2, 3, 32)
    assert torch.equal(packed & 15, codes[..., 0::2]) and torch.equal(packed >> 4, codes[..., 1::2])


def test_empty_batches_are_no_ops(moe):
    assert back(moe, T=0, rows=None, offsets=None, e2s=None, out=None) == 0
    assert grad(moe, T=0, dout=None, rows=None, offsets=None, e2s=None, w=None, drows=None,
                dw=None) == 0
    assert moe.lib.moe_sort_tokens_backward(0, 2, 8, 64, BF16, None, None, None, FP32, None, 64,
                                            None) == 0


def test_binding_checks_tensors_before_the_library(moe):
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="current CUDA device"):
        moe.moe_add_rmsnorm(x, None, None, 1e-6, x)
    with pytest.raises(TypeError, match="x"):
        moe.moe_add_rmsnorm(x.double(), None, None, 1e-6, x)
    with pytest.raises(TypeError, match="matrix"):
        moe.moe_add_rmsnorm(x[0], None, None, 1e-6, x)
    with pytest.raises(ValueError, match="not contiguous"):
        moe.moe_add_rmsnorm(x[:, ::2], None, None, 1e-6, x)
    ids = torch.zeros(4, 2, dtype=torch.int64)
    with pytest.raises(TypeError, match="ids"):
        moe.moe_sort_tokens(8, ids, None, None, None, None, None, None, None)


def test_binding_refuses_to_write_what_requires_a_gradient(moe):
    # before anything is launched, and whatever the device
    x, out = torch.zeros(4, 64), torch.zeros(4, 64, requires_grad=True)
    with pytest.raises(ValueError, match="sum_out: requires a gradient"):
        moe.moe_add_rmsnorm(x, None, None, 1e-6, out)
    with pytest.raises(ValueError, match="y: requires a gradient"):
        moe.moe_add_rmsnorm(x, None, None, 1e-6, x, out)
    i32 = dict(dtype=torch.int32)
    with pytest.raises(ValueError, match="out: requires a gradient"):
        moe.moe_unsort_tokens(torch.zeros(8, 64), torch.zeros(9, **i32), torch.zeros(8, **i32),
                              torch.zeros(4, 2), out)
    with torch.no_grad(), pytest.raises(ValueError, match="current CUDA device"):
        moe.moe_add_rmsnorm(x, None, None, 1e-6, out)


def test_binding_names_what_is_not_a_tensor(moe):
    i32 = dict(dtype=torch.int32)
    x, rows, w, bad = torch.zeros(4, 64), torch.zeros(8, 64), torch.zeros(4, 2), [1.0]
    ids = torch.zeros(4, 2, **i32)
    plan = [torch.zeros(n, **i32) for n in (8, 9, 8, 8)]
    u8 = torch.zeros(1, 8, 32, dtype=torch.uint8)
    calls = [
        ("x", lambda: moe.moe_sort_tokens(8, ids, bad, None, *plan, rows)),
        ("x_sorted", lambda: moe.moe_sort_tokens(8, ids, x, None, *plan, bad)),
        ("x_scale", lambda: moe.moe_sort_tokens(8, ids, x, bad, *plan, rows, w)),
        ("scale_sorted", lambda: moe.moe_sort_tokens(8, ids, x, x[:, 0].clone(), *plan, rows, bad)),
        ("ws", lambda: moe.moe_sort_tokens(8, ids, x, None, *plan, rows, None, bad)),
        ("offsets", lambda: moe.moe_sort_tokens_backward(rows, bad, plan[3], 2, x)),
        ("expanded_to_sorted", lambda: moe.moe_sort_tokens_backward(rows, plan[1], bad, 2, x)),
        ("topk_w", lambda: moe.moe_unsort_tokens(rows, plan[1], plan[3], bad, x)),
        ("topk_w", lambda: moe.moe_unsort_tokens(rows, plan[1], plan[3], w[0, 0], x)),
        ("topk_w", lambda: moe.moe_unsort_tokens_backward(x, rows, plan[1], plan[3], bad, rows, w)),
        ("offsets", lambda: moe.moe_unsort_tokens_backward(x, rows, None, plan[3], w, rows, w)),
        ("x_scale", lambda: moe.moe_w4_gemv(x.bfloat16(), bad, None, u8, torch.ones(1, 8, 1), None,
                                            torch.zeros(4, 8))),
    ]
    for name, call in calls:
        with pytest.raises(TypeError, match=f"^{name}: "):
            call()
