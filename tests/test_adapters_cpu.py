"""moe_adapters and moe_adapters_backward refuse bad arguments on the host, before any
launch."""
import ctypes

import pytest

FAKE = 1 << 40  # never dereferenced
BF16, FP16, FP32, INT8 = 0, 1, 2, 3
INVALID, UNSUPPORTED, ALIGNMENT, WS = 1, 2, 3, 4


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__

    __graft_entry__._builder().build()
    import sparse_expert_layer_gb300 as m

    return m


def forward(moe, **kw):
    a = dict(T=4, J=2, r=16, K=64, N=128, dtype=BF16, x=FAKE, ldx=64, a=FAKE, b=FAKE, scale=FAKE,
             offsets=FAKE, order=FAKE, base=FAKE, ldb=128, y=FAKE + 4096, ldy=128, v=FAKE, ws=FAKE,
             ws_bytes=1 << 30)
    a.update(kw)
    return moe.lib.moe_adapters(*a.values(), None)


def backward(moe, **kw):
    a = dict(T=4, J=2, r=16, K=64, N=128, dtype=BF16, dy=FAKE, lddy=128, x=FAKE, ldx=64, v=FAKE,
             a=FAKE, b=FAKE, scale=FAKE, offsets=FAKE, order=FAKE, dx=FAKE + 4096, lddx=64,
             grad_dtype=FP32, da=FAKE, db=FAKE, ws=FAKE, ws_bytes=1 << 30)
    a.update(kw)
    return moe.lib.moe_adapters_backward(*a.values(), None)


COMMON = [(dict(T=-1), INVALID), (dict(J=0), INVALID), (dict(r=0), INVALID), (dict(K=0), INVALID),
          (dict(N=0), INVALID), (dict(dtype=FP32), INVALID), (dict(dtype=INT8), INVALID),
          (dict(r=129), UNSUPPORTED), (dict(J=4097), UNSUPPORTED),
          (dict(T=(1 << 21) + 1), UNSUPPORTED), (dict(ldx=63), INVALID), (dict(a=None), INVALID),
          (dict(b=None), INVALID), (dict(offsets=None), INVALID), (dict(ws=None), INVALID),
          (dict(ws_bytes=100), WS), (dict(ws=FAKE + 128), ALIGNMENT), (dict(x=FAKE + 2), ALIGNMENT),
          (dict(a=FAKE + 8), ALIGNMENT), (dict(b=FAKE + 8), ALIGNMENT),
          (dict(scale=FAKE + 4), ALIGNMENT), (dict(offsets=FAKE + 4), ALIGNMENT),
          (dict(order=FAKE + 4), ALIGNMENT), (dict(v=FAKE + 4), ALIGNMENT)]


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(x=None), INVALID), (dict(y=None), INVALID), (dict(ldy=127), INVALID),
    (dict(ldb=127), INVALID), (dict(y=FAKE, ldy=136), INVALID), (dict(y=FAKE + 2), ALIGNMENT),
    (dict(base=FAKE + 2), ALIGNMENT), (dict(x=FAKE + 4096), INVALID), (dict(K=(1 << 21) + 1, ldx=1 << 22), UNSUPPORTED),
    (dict(N=(1 << 21) + 1, ldb=1 << 22, ldy=1 << 22), UNSUPPORTED)])
def test_refusals(moe, kw, status):
    assert forward(moe, **kw) == status


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(dy=None), INVALID), (dict(x=None), INVALID), (dict(v=None), INVALID),
    (dict(lddy=127), INVALID), (dict(lddx=63), INVALID), (dict(da=None), INVALID),
    (dict(db=None), INVALID), (dict(dx=None, da=None, db=None), INVALID),
    (dict(dx=FAKE), INVALID), (dict(dy=FAKE + 4096), INVALID), (dict(grad_dtype=FP16), INVALID), (dict(grad_dtype=INT8), INVALID),
    (dict(da=FAKE + 4), ALIGNMENT), (dict(dx=FAKE + 4), ALIGNMENT), (dict(dy=FAKE + 4), ALIGNMENT)])
def test_backward_refusals(moe, kw, status):
    assert backward(moe, **kw) == status


def test_no_rows_is_a_no_op(moe):
    assert forward(moe, T=0, x=None, y=None, ws=None) == 0
    assert backward(moe, T=0, dy=None, da=None, db=None) == 0


def test_workspace_size(moe):
    a, b = (moe.moe_adapters_workspace_size(T, 16, 64, 128) for T in (64, 8192))
    assert 64 * 16 * 4 <= a < b
    n = ctypes.c_size_t(0)
    assert moe.lib.moe_adapters_workspace_size(-1, 16, 64, 64, ctypes.byref(n)) == INVALID
    assert moe.lib.moe_adapters_workspace_size(4, 129, 64, 64, ctypes.byref(n)) == UNSUPPORTED
    assert moe.lib.moe_adapters_workspace_size(4, 16, 64, 64, None) == INVALID
    assert moe.adapters_workspace(4, 16, 64, 128, "cpu").numel() > 0


def test_a_scale_that_wants_a_gradient_is_refused(moe):
    import torch

    from sparse_expert_layer_gb300 import autograd

    x, a, b = torch.zeros(4, 64), torch.zeros(2, 16, 64), torch.zeros(2, 16, 128)
    plan = autograd.SortPlan(*(torch.zeros(4, dtype=torch.int32) for _ in range(4)))
    with pytest.raises(RuntimeError, match="scale"):
        autograd.adapters(None, x, a, b, torch.ones(2, requires_grad=True), plan)


def test_a_scale_that_wants_a_gradient_is_a_constant_under_no_grad(moe):
    import torch

    from sparse_expert_layer_gb300 import autograd

    x, a, b = (torch.zeros(*s, dtype=torch.bfloat16) for s in ((4, 64), (2, 16, 64), (2, 16, 128)))
    plan = autograd.SortPlan(*(torch.zeros(n, dtype=torch.int32) for n in (2, 3, 4, 4)))
    # (as far as the launch, for which these tensors are on the wrong device)
    with torch.no_grad(), pytest.raises(ValueError, match="not on the current CUDA device"):
        autograd.adapters(None, x, a, b, torch.ones(2, requires_grad=True), plan)


@pytest.mark.parametrize("layout", ["slice", "column"])
def test_a_scale_of_another_layout_is_copied(moe, monkeypatch, layout):
    import torch

    from sparse_expert_layer_gb300 import autograd

    seen = []
    monkeypatch.setattr(autograd.ops, "moe_adapters", lambda x, a, b, scale, *rest: seen.append(scale))
    x, a, b = (torch.zeros(*s, dtype=torch.bfloat16) for s in ((4, 64), (2, 16, 64), (2, 16, 128)))
    plan = autograd.SortPlan(*(torch.zeros(n, dtype=torch.int32) for n in (2, 3, 4, 4)))
    scale = {"slice": torch.arange(5.0)[1:3], "column": torch.arange(8.0).view(2, 4)[:, 1]}[layout]
    autograd.adapters(None, x, a, b, scale, plan)
    (got,) = seen
    assert torch.equal(got, scale) and got.is_contiguous() and got.data_ptr() % 16 == 0
