"""moe_few_tokens refuses bad arguments on the host, before any launch."""
import ctypes

import pytest
import torch

FAKE = 1 << 40  # never dereferenced
BF16, FP16, FP32, INT8, U4 = 0, 1, 2, 3, 5
INVALID, UNSUPPORTED, ALIGNMENT, WS = 1, 2, 3, 4


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__

    __graft_entry__._builder().build()
    import sparse_expert_layer_gb300 as m

    return m


def config(moe, **kw):
    spec = dict(hidden=256, inter=128, n_routed=8, top_k=2, shared_inter=64, bias_mode="logit")
    spec.update(kw)
    return moe.config_from_spec(spec)


def weights(moe, four, **kw):
    a = dict(w_dtype=U4 if four else BF16, group=32, scale_dtype=BF16, w=FAKE, scales=FAKE,
             zeros=None, shared_zeros=None, part="routed", at=0)
    a.update(kw)
    c = moe.MoeFewWeights(a["w_dtype"], a["group"], a["scale_dtype"])
    for part in (c.routed, c.shared):
        for i in range(3):
            part.w[i] = FAKE
            part.scales[i] = FAKE if four else None
    for i in range(3):
        c.routed.zeros[i], c.shared.zeros[i] = a["zeros"], a["shared_zeros"]
    p = getattr(c, a["part"])
    p.w[a["at"]] = a["w"]
    if four or a["scales"] != FAKE:
        p.scales[a["at"]] = a["scales"]
    return c


def call(moe, four=False, cfg=None, wt=None, **kw):
    a = dict(T=4, dtype=BF16, x=FAKE, ldx=256, w_router=FAKE, bias=FAKE, ids=None, w=None,
             out=FAKE + 4096, ldo=256, ws=FAKE, ws_bytes=1 << 40)
    a.update(kw)
    return moe.lib.moe_few_tokens(ctypes.byref(config(moe, **(cfg or {}))),
                                  ctypes.byref(weights(moe, four, **(wt or {}))), *a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INVALID), (dict(out=FAKE), INVALID),
    (dict(cfg=dict(inter=(1 << 20) + 32)), UNSUPPORTED),
    (dict(cfg=dict(shared_inter=(1 << 20) + 32)), UNSUPPORTED), (dict(T=9), UNSUPPORTED), (dict(dtype=FP32), INVALID),
    (dict(dtype=FP16), INVALID), (dict(x=None), INVALID), (dict(ldx=255), INVALID),
    (dict(w_router=None), INVALID), (dict(bias=None), INVALID), (dict(out=None), INVALID),
    (dict(ldo=100), INVALID), (dict(ws=None), INVALID), (dict(ws_bytes=1000), WS),
    (dict(x=FAKE + 2), ALIGNMENT), (dict(out=FAKE + 8), ALIGNMENT), (dict(ws=FAKE + 16), ALIGNMENT),
    (dict(ids=FAKE + 4), ALIGNMENT), (dict(w=FAKE + 4), ALIGNMENT), (dict(bias=FAKE + 4), ALIGNMENT),
    (dict(w_router=FAKE + 4), ALIGNMENT), (dict(wt=dict(w=None)), INVALID),
    (dict(wt=dict(w=None, part="shared", at=2)), INVALID), (dict(wt=dict(w=FAKE + 2)), ALIGNMENT),
    (dict(wt=dict(scales=FAKE + 16)), INVALID), (dict(wt=dict(w_dtype=INT8)), INVALID),
    (dict(cfg=dict(wdtype="w8a8")), UNSUPPORTED), (dict(cfg=dict(hidden=7)), INVALID),
    (dict(cfg=dict(top_k=9)), INVALID), (dict(T=8, cfg=dict(hidden=8200), ldx=8200, ldo=8200),
                                         UNSUPPORTED),
])
def test_refusals(moe, kw, status):
    assert call(moe, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(wt=dict(group=48)), INVALID), (dict(wt=dict(group=-32)), INVALID),
    (dict(wt=dict(scale_dtype=INT8)), INVALID), (dict(wt=dict(scales=None)), INVALID),
    (dict(wt=dict(scales=None, part="shared", at=1)), INVALID),
    (dict(wt=dict(scales=FAKE + 2)), ALIGNMENT), (dict(wt=dict(zeros=FAKE)), INVALID),
    (dict(wt=dict(shared_zeros=FAKE)), INVALID),
    (dict(wt=dict(zeros=FAKE + 1, shared_zeros=FAKE)), ALIGNMENT),
    (dict(wt=dict(group=128)), INVALID),  # the shared expert's 64 is no multiple of it
    (dict(cfg=dict(hidden=264), ldx=264, ldo=264), INVALID), (dict(cfg=dict(inter=72)), INVALID),
    (dict(cfg=dict(shared_inter=40)), INVALID), (dict(dtype=FP32), INVALID),
])
def test_four_bit_refusals(moe, kw, status):
    assert call(moe, four=True, **kw) == status


def test_no_tokens_is_a_no_op(moe):
    assert call(moe, T=0, x=None, out=None, ws=None) == 0
    assert call(moe, four=True, T=0, x=None, out=None, ws=None) == 0
    assert moe.lib.moe_few_tokens(ctypes.byref(config(moe)), None, 0, BF16, None, 256, None, None,
                                  None, None, None, 256, None, 0, None) == INVALID
    assert moe.lib.moe_few_tokens(None, None, 0, BF16, None, 256, None, None, None, None, None,
                                  256, None, 0, None) == INVALID


def test_workspace_size(moe):
    sizes = [moe.moe_few_tokens_workspace_size(config(moe), T) for T in (1, 4, 8)]
    assert 0 < sizes[0] < sizes[1] < sizes[2]
    for T in (-1, 9):
        with pytest.raises(moe.MoeError):
            moe.moe_few_tokens_workspace_size(config(moe), T)
    n = ctypes.c_size_t(0)
    assert moe.lib.moe_few_tokens_workspace_size(None, 1, ctypes.byref(n)) == INVALID
    assert moe.lib.moe_few_tokens_workspace_size(ctypes.byref(config(moe)), 1, None) == INVALID


@pytest.mark.parametrize("T", [1, 2, 8])
def test_an_inter_that_no_expert_has_changes_nothing(moe, T):
    # rows of h are the shared expert's then: whole 16-byte pieces, whatever inter is
    sizes = {moe.moe_few_tokens_workspace_size(
        config(moe, n_routed=0, n_zero=4, inter=inter, shared_inter=8), T)
        for inter in (0, 8, 50, 4097, (1 << 20) + 3)}
    assert len(sizes) == 1
    # inter of routed experts is that of h, and checked
    with pytest.raises(moe.MoeError):
        moe.moe_few_tokens_workspace_size(config(moe, inter=50), T)


def handle(moe, four=False, drop=(), cfg=None, **kw):
    """A FewTokenExperts of CPU tensors (never launched)."""
    c = config(moe, **(cfg or {}))
    w = {}
    for prefix, infix, lead, inter in (("w_", "", (8,), 128), ("shared_", "shared_", (), 64)):
        for mat, n, k in (("gate", inter, 256), ("up", inter, 256), ("down", 256, inter)):
            w[prefix + mat] = torch.zeros(*lead, n, k // 2, dtype=torch.uint8) if four else \
                torch.zeros(*lead, n, k, dtype=torch.bfloat16)
            if four:
                w[f"s_{infix}{mat}"] = torch.ones(*lead, n, k // 32, dtype=torch.bfloat16)
    w.update(kw)
    for d in drop:
        del w[d]
    return moe.FewTokenExperts(c, w, torch.zeros(8, 256), torch.zeros(8))


def test_handles_are_checked(moe):
    assert handle(moe).dtype == torch.bfloat16
    four = handle(moe, True)
    assert four.dtype is None and four.c.group == 32 and four.c.scale_dtype == BF16
    with pytest.raises(TypeError, match="cfg"):
        moe.FewTokenExperts({}, {}, torch.zeros(8, 256))
    with pytest.raises(TypeError, match="w_up"):
        handle(moe, drop=["w_up"])
    with pytest.raises(TypeError, match="shared_down"):
        handle(moe, drop=["shared_down"])
    with pytest.raises(TypeError, match="w_up: torch.float16"):
        handle(moe, w_up=torch.zeros(8, 128, 256, dtype=torch.float16))
    with pytest.raises(ValueError, match="w_down: shape"):
        handle(moe, w_down=torch.zeros(8, 128, 256, dtype=torch.bfloat16))
    with pytest.raises(TypeError, match="weights: torch.float32"):
        handle(moe, w_gate=torch.zeros(8, 128, 256))
    with pytest.raises(TypeError, match="s_gate"):
        handle(moe, True, drop=["s_gate"])
    with pytest.raises(ValueError, match="s_up: groups of 64"):
        handle(moe, True, s_up=torch.ones(8, 128, 4, dtype=torch.bfloat16))
    with pytest.raises(TypeError, match="s_up: torch.float32"):
        handle(moe, True, s_up=torch.ones(8, 128, 8))
    with pytest.raises(ValueError, match="zero points for all"):
        handle(moe, True, z_up=torch.ones(8, 128, 8, dtype=torch.uint8))
    with pytest.raises(ValueError, match="s_shared_down: 3 groups"):
        handle(moe, True, s_shared_down=torch.ones(256, 3, dtype=torch.bfloat16))
    x = torch.zeros(2, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="not on the current CUDA device"):
        moe.moe_few_tokens(four, x, x.clone(), torch.zeros(1 << 20, dtype=torch.uint8))


def test_a_description_that_changes_later_changes_no_handle(moe, monkeypatch):
    # the sizes that the weights were checked against stay those of every call
    made = []
    monkeypatch.setitem(globals(), "config", lambda *a, _c=config, **kw: made.append(_c(*a, **kw))
                        or made[-1])
    experts = handle(moe)
    size = moe.few_tokens_workspace(experts, 4).numel()
    made[-1].hidden, made[-1].inter, made[-1].n_routed, made[-1].top_k = 512, 256, 16, 4
    assert (experts.cfg.hidden, experts.cfg.inter, experts.cfg.n_routed, experts.cfg.top_k) == \
        (256, 128, 8, 2)
    assert moe.few_tokens_workspace(experts, 4).numel() == size
