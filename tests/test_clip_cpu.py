"""moe_clip_grad_norm refuses bad arguments on the host, before any launch."""
import ctypes

import pytest
import torch

FAKE = 1 << 40  # never dereferenced
BF16, FP16, FP32, INT8 = 0, 1, 2, 3
INVALID, UNSUPPORTED, ALIGNMENT, WS = 1, 2, 3, 4


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__

    __graft_entry__._builder().build()
    import sparse_expert_layer_gb300 as m

    return m


def call(moe, tensor=None, **kw):
    t = dict(in_=FAKE, out=FAKE, n=10, dtype=FP32)
    t.update(tensor or {})
    a = dict(n=1, tensors=(moe.MoeTensor * 1)(moe.MoeTensor(**t)), max_norm=1.0, eps=1e-6,
             norm=FAKE, ws=FAKE, ws_bytes=1 << 20)
    a.update(kw)
    return moe.lib.moe_clip_grad_norm(*a.values(), None)


@pytest.mark.parametrize("tensor,kw,status", [
    (None, dict(n=-1), INVALID), (None, dict(tensors=None), INVALID),
    (None, dict(max_norm=-1.0), INVALID), (None, dict(max_norm=float("nan")), INVALID),
    (None, dict(max_norm=float("inf")), INVALID), (None, dict(eps=-1e-6), INVALID),
    (None, dict(eps=float("nan")), INVALID), (None, dict(ws=None), INVALID),
    (None, dict(ws=FAKE + 128), ALIGNMENT), (None, dict(ws_bytes=100), WS),
    (None, dict(norm=FAKE + 2), ALIGNMENT), (dict(n=-1), {}, INVALID),
    (dict(dtype=INT8), {}, INVALID), (dict(dtype=-1), {}, INVALID), (dict(in_=None), {}, INVALID),
    (dict(in_=FAKE + 2), {}, ALIGNMENT), (dict(out=FAKE + 2), {}, ALIGNMENT),
    (dict(in_=FAKE + 1, dtype=BF16), {}, ALIGNMENT), (dict(n=1 << 43), {}, UNSUPPORTED),
    (dict(out=None), dict(norm=None), INVALID), (None, dict(n=0, norm=None), INVALID),
])
def test_refusals(moe, tensor, kw, status):
    assert call(moe, tensor, **kw) == status


def test_workspace_size(moe):
    assert moe.moe_clip_workspace_size() > 0
    assert moe.lib.moe_clip_workspace_size(None) == INVALID
    assert moe.clip_workspace("cpu").numel() == moe.moe_clip_workspace_size()
    assert ctypes.sizeof(moe.MoeTensor) == 32


def test_lists_are_checked(moe, monkeypatch):
    from sparse_expert_layer_gb300 import operators

    with pytest.raises(TypeError, match=r"tensors\[1\]: expected a tensor"):
        operators.TensorList([torch.zeros(3), 4.0])
    with pytest.raises(ValueError, match="outs: 1 for 2"):
        operators.TensorList([torch.zeros(3), torch.zeros(3)], [torch.zeros(3)])
    with pytest.raises(TypeError, match=r"tensors\[0\]: torch.int8"):
        operators.TensorList([torch.zeros(3, dtype=torch.int8)])
    with pytest.raises(ValueError, match="not contiguous"):
        operators.TensorList([torch.zeros(4, 4).t()])
    with pytest.raises(ValueError, match=r"outs\[0\]: shape"):
        operators.TensorList([torch.zeros(4)], [torch.zeros(5)])
    with pytest.raises(TypeError, match=r"outs\[0\]"):
        operators.TensorList([torch.zeros(4)], [torch.zeros(4, dtype=torch.bfloat16)])
    t = torch.zeros(100)
    for tensors, outs in (([t, t], None), ([t[:60], t[50:]], None), ([t[:50]], [t[1:51]]),
                          ([t[:50], t[50:]], [t[50:], None])):
        with pytest.raises(ValueError, match="overlaps"):
            operators.TensorList(tensors, outs)
    operators.TensorList([t[:50], t[50:]])
    operators.TensorList([t, t[10:20], t], [None, None, None])  # only counted: read twice
    operators.TensorList([t[:0], t, t[5:5]])
    with pytest.raises(ValueError, match="not on the current CUDA device"):
        operators.moe_clip_grad_norm([t], 1.0, None, operators.clip_workspace("cpu"))


def test_no_tensors_and_no_workspace(moe):
    with pytest.raises(TypeError, match="ws: expected a tensor"):
        moe.moe_clip_grad_norm([], 1.0, None, None)
    with pytest.raises(ValueError, match="not on the current CUDA device"):
        moe.moe_clip_grad_norm([], 1.0, torch.zeros(1), moe.clip_workspace("cpu"))
