"""moe_few_tokens against its definition: picks and weights from the fp64 oracle's
router, the experts in 64 bits on the GPU.

Tolerance, element by element, u = 2^-24.  A sum of K products leaves at most
(K / 8 + 64) u times the sum of the magnitudes that were added: each MMA of sixteen
products rounds within two u of what it holds, and the few additions that join blocks,
warps and scales follow (4 bits: the magnitudes are those of q x and z x).  h carries
the errors of gate and up (|silu'| <= 1.1) and its own rounding: 2^-12 of it and 2^-34
of the row's largest with 4-bit weights, 2^-17 as two bf16 numbers, 2^-22 as two fp16
ones.  Routing weights are within 1e-5, and out is rounded once.
"""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import oracle
import synth
from tests import gpu_support as gs
from tests import support

pytestmark = pytest.mark.gpu

U = 2.0**-24
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
TINY = {BF16: 2.0**-134, FP16: 2.0**-25}
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def m():
    return gs.lib()


def gen(seed=0):
    return torch.Generator(device="cuda").manual_seed(seed)


# description overrides of a small softmax layer
LAYERS = {
    "flat": dict(hidden=512, inter=256, n_routed=16, top_k=4, renormalize=True),
    "groups": dict(hidden=1024, inter=320, n_routed=64, top_k=8, n_group=8, topk_group=4,
                   score="sigmoid", renormalize=True, routed_scale=2.5, shared_inter=384),
    "per_group": dict(hidden=640, inter=384, n_routed=64, top_k=8, n_group=8, per_group_k=1,
                      shared_inter=512),
    "zero": dict(hidden=1024, inter=384, n_routed=96, n_zero=48, top_k=12, bias_mode="logit",
                 bias_kind="iid", renormalize=False),
    "select": dict(hidden=288, inter=96, n_routed=24, top_k=3, score="sigmoid",
                   bias_mode="select", bias_kind="iid", renormalize=True),
    "only_zero": dict(hidden=256, inter=32, n_routed=0, n_zero=8, top_k=2, renormalize=True),
    "only_shared": dict(hidden=256, inter=32, n_routed=0, n_zero=4, top_k=1, shared_inter=160),
    "all": dict(hidden=160, inter=64, n_routed=32, top_k=32, renormalize=True),
    "one": dict(hidden=32, inter=32, n_routed=1, top_k=1),
    "flat256": dict(hidden=64, inter=32, n_routed=250, top_k=9, renormalize=True),
    "flat512": dict(hidden=96, inter=32, n_routed=300, n_zero=200, top_k=32, bias_mode="logit",
                    bias_kind="iid"),
    "flat768": dict(hidden=64, inter=32, n_routed=513, top_k=7, score="sigmoid",
                    bias_mode="select", bias_kind="iid"),
    "flat1024": dict(hidden=64, inter=32, n_routed=1024, top_k=5, routed_scale=1.5),
    "groups_wide": dict(hidden=64, inter=32, n_routed=1600, top_k=4, n_group=8, topk_group=3),
    "wide": dict(hidden=64, inter=32, n_routed=2048, top_k=6),
    "deep": dict(hidden=7168, inter=2048, n_routed=12, top_k=4, shared_inter=2048),
    # 16-bit weights only
    "ragged": dict(hidden=1000, inter=200, n_routed=24, n_zero=8, top_k=5, bias_mode="logit",
                   bias_kind="iid", shared_inter=136),
    "eight": dict(hidden=8, inter=8, n_routed=4, top_k=2, shared_inter=8),
    "more_channels": dict(hidden=13104, inter=48, n_routed=4, top_k=2),
}


def make(name, T, dtype, bits, group=0, zeros=False, sdt=None, seed=0):
    """A layer's inputs: description, x, router, bias and weights on the GPU."""
    spec = synth.spec("tiny", T=T, name=f"few_{name}", **dict(
        dict(n_zero=0, renormalize=False), **LAYERS[name]))
    x, w_r, bias, _ = support.make_inputs(spec, seed)
    # values that both 16-bit types hold
    x = torch.where(x.abs() < 2.0**-16, torch.zeros_like(x), x)
    g = gen(seed + T)
    E, H, I, Is = spec["n_routed"], spec["hidden"], spec["inter"], spec["shared_inter"]
    w = {}

    def stack(key, infix, mat, shape):
        K = shape[-1]
        if bits == 16:
            w[key] = (torch.randn(*shape, generator=g, device="cuda") / K**0.5).to(dtype)
            return
        groups = K // group if group else 1
        codes = torch.randint(0, 16, shape, generator=g, device="cuda", dtype=torch.uint8)
        w[key] = gs.lib().pack_w4(codes)
        w[f"s_{infix}{mat}"] = ((0.3 + torch.rand(*shape[:-1], groups, generator=g, device="cuda"))
                                / (4.6 * K**0.5)).to(sdt or dtype)
        if zeros:
            w[f"z_{infix}{mat}"] = torch.randint(0, 32, (*shape[:-1], groups), generator=g,
                                                 device="cuda", dtype=torch.uint8)

    for mat, n, k in (("gate", I, H), ("up", I, H), ("down", H, I)):
        if E:
            stack("w_" + mat, "", mat, (E, n, k))
        if Is:
            n, k = (Is if mat != "down" else H), (H if mat != "down" else Is)
            stack("shared_" + mat, "shared_", mat, (n, k))
    return dict(spec=spec, x16=x, x=x.to(dtype).cuda(), w_r=w_r, bias=bias, w=w, bits=bits,
                dtype=dtype)


def exact_matrix(w, key, infix, mat, e):
    """(values, magnitudes that the kernel adds) of one matrix in 64 bits."""
    t = w[key] if e is None else w[key][e]
    if t.dtype != torch.uint8:
        v = t.double()
        return v, v.abs()
    s = w[f"s_{infix}{mat}"]
    z = w.get(f"z_{infix}{mat}")
    s, z = (s, z) if e is None else (s[e], None if z is None else z[e])
    q = torch.stack([t & 15, t >> 4], -1).view(t.shape[0], -1).double()
    width = q.shape[1] // s.shape[1]
    z = torch.full_like(s, 8.0, dtype=torch.float64) if z is None else z.double()
    z, s = z.repeat_interleave(width, 1), s.double().repeat_interleave(width, 1)
    return (q - z) * s, (q + z) * s


def exact_ffn(c, prefix, infix, e, x):
    """(y, bound of its error) of one expert for one token, in 64 bits."""
    four = c["bits"] == 4

    def product(mat, v, mag):
        a, b = exact_matrix(c["w"], prefix + mat, infix, mat, e)
        return a @ v, (a.shape[1] / 8 + 64) * U * (b @ mag), a

    xa = x.abs()
    # 4 bits: x below 2^-23 of its largest is rounded at 2^-33 of that
    round_x = 2.0**-33 * xa.max() if four else 0.0
    g, dg, ga = product("gate", x, xa)
    u, du, ua = product("up", x, xa)
    dg = dg + round_x * ga.abs().sum(1)
    du = du + round_x * ua.abs().sum(1)
    silu = g * torch.sigmoid(g)
    h = silu * u
    dh = 1.1 * dg * u.abs() + (silu.abs() + 1.1 * dg) * du + 16 * U * h.abs()
    top = (h.abs() + dh).max()
    rel = 2.0**-12 if four else 2.0**-17 if c["dtype"] == BF16 else 2.0**-22
    dh = dh + rel * (h.abs() + dh) + 2.0**-34 * top
    y, dy, da = product("down", h, h.abs() + dh)
    return y, dy + da.abs() @ dh


def exact(c, ids, wts):
    """(out, bound) of the whole layer; ids, wts [T, k] in 64 bits."""
    spec = c["spec"]
    E = spec["n_routed"]
    T = ids.shape[0]
    out = torch.zeros(T, spec["hidden"], dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(out)
    for t in range(T):
        x = c["x"][t].double()
        for e, p in zip(ids[t].tolist(), wts[t].tolist()):
            y, dy = exact_ffn(c, "w_", "", e, x) if e < E else (x, torch.zeros_like(x))
            out[t] += p * y
            tol[t] += abs(p) * (dy + (1e-5 + 64 * U) * y.abs())
        if spec["shared_inter"]:
            y, dy = exact_ffn(c, "shared_", "shared_", None, x)
            out[t] += y
            tol[t] += dy + 64 * U * y.abs()
    return out, tol + torch.finfo(c["dtype"]).eps / 2 * (out.abs() + tol) + TINY[c["dtype"]]


def experts_of(m, c):
    cfg = m.config_from_spec(c["spec"])
    bias = None if c["bias"] is None else c["bias"].cuda()
    return m.FewTokenExperts(cfg, c["w"], c["w_r"].cuda(), bias)


def routed(c):
    spec = c["spec"]
    ids, w, _, _ = oracle.route(spec, synth.bf16_bits(c["x16"]), c["w_r"].numpy(),
                                support.np_bias(c["bias"]))
    return torch.from_numpy(np.asarray(ids)), torch.from_numpy(np.asarray(w, dtype=np.float64))


def check(m, c, x=None, extra=0):
    spec = c["spec"]
    T, H, k = spec["T"], spec["hidden"], spec["top_k"]
    experts = experts_of(m, c)
    ws = m.few_tokens_workspace(experts, T)
    guard = torch.full((ws.numel() + 512,), 0, dtype=torch.uint8, device="cuda")
    guard[ws.numel():] = 99
    x = c["x"] if x is None else x
    wide = torch.full((T, H + extra), 7.0, dtype=c["dtype"], device="cuda")
    ids = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), -1.0, device="cuda")
    m.moe_few_tokens(experts, x, wide[:, :H], guard[:ws.numel()], ids, w)
    torch.cuda.synchronize()
    assert m.moe_check_device_status(guard) == m.MOE_OK
    assert (guard[ws.numel():] == 99).all() and (wide[:, H:] == 7).all()
    ids_o, w_o = routed(c)
    assert torch.equal(ids.cpu().long(), ids_o.long())
    assert np.allclose(w.cpu().numpy(), w_o.numpy(), rtol=1e-5, atol=1e-7)
    want, tol = exact(c, ids_o, w_o)
    over = (wide[:, :H].double() - want).abs() - tol
    assert float(over.max()) <= 0, f"off by {float((wide[:, :H].double() - want).abs().max()):.3e}, " \
        f"{float(over.max()):.3e} more than allowed"
    return wide[:, :H]


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("T", [1, 2, 3, 8])
@pytest.mark.parametrize("name", list(LAYERS))
def test_sixteen_bit_weights(m, name, T, dtype):
    if T * LAYERS[name]["hidden"] > 65536:
        T = 65536 // LAYERS[name]["hidden"]
    check(m, make(name, T, dtype, 16))


FOUR = ["flat", "flat512", "flat768", "groups", "per_group", "zero", "select", "only_zero", "only_shared", "all", "one",
        "wide", "deep"]


@pytest.mark.parametrize("T", [1, 2, 5, 8])
@pytest.mark.parametrize("name", FOUR)
@pytest.mark.parametrize("dtype,group,zeros,sdt", [(BF16, 32, False, BF16), (BF16, 0, True, FP32),
                                                   (FP16, 32, True, FP16), (FP16, 0, False, BF16)])
def test_four_bit_weights(m, name, T, dtype, group, zeros, sdt):
    check(m, make(name, T, dtype, 4, group, zeros, sdt))


@pytest.mark.parametrize("T", [1, 4, 8])
@pytest.mark.parametrize("name,group", [("flat", 64), ("flat", 128), ("per_group", 128),
                                        ("groups", 64), ("zero", 64), ("zero", 128),
                                        ("deep", 64), ("deep", 128), ("deep", 32)])
@pytest.mark.parametrize("zeros,sdt", [(False, BF16), (True, FP16), (True, FP32)])
def test_four_bit_groups(m, name, T, group, zeros, sdt):
    check(m, make(name, T, BF16, 4, group, zeros, sdt))


@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("T", [2, 3, 7])
def test_all_tokens_alike(m, bits, T):
    # every expert has all tokens
    c = make("groups", T, BF16, bits, 32)
    c["x16"][:] = c["x16"][0].clone()
    c["x"][:] = c["x"][0].clone()
    out = check(m, c)
    assert (out == out[0]).all()


@pytest.mark.parametrize("extra", [8, 3])
@pytest.mark.parametrize("bits", [4, 16])
def test_row_strides(m, extra, bits):
    c = make("flat", 5, BF16, bits, 64)
    wide = torch.full((5, 512 + extra), float("nan"), dtype=BF16, device="cuda")
    wide[:, :512] = c["x"]
    check(m, c, wide[:, :512], extra)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("bits", [4, 16])
def test_a_loud_channel(m, dtype, bits):
    # x spans many binades; its largest value sets the scale of a 4-bit product's x
    c = make("flat", 3, dtype, bits, 32)
    scale = torch.exp2(torch.randint(-12, 1, c["x"].shape, generator=gen(1), device="cuda").float())
    x = (c["x"].float() * scale).to(BF16)
    x[:, 17] *= 64
    x = torch.where(x.abs() < 2.0**-16, torch.zeros_like(x), x)
    c["x16"], c["x"] = x.cpu(), x.to(dtype)
    if not support.margin_rows(c["spec"], c["x16"], c["w_r"], c["bias"], 1e-4).all():
        pytest.skip("the picks are not clear")
    check(m, c)


@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_token_that_is_not_finite_stays_alone(m, bits, bad):
    c = make("flat", 4, BF16, bits, 32)
    experts = experts_of(m, c)
    ws = m.few_tokens_workspace(experts, 4)
    good, out = torch.empty_like(c["x"]), torch.empty_like(c["x"])
    m.moe_few_tokens(experts, c["x"], good, ws)
    x = c["x"].clone()
    x[2, 5] = bad
    m.moe_few_tokens(experts, x, out, ws)
    torch.cuda.synchronize()
    rest = [0, 1, 3]
    # (the other token's picks may differ, and with them the order of the sums)
    assert torch.isfinite(out[rest]).all()
    assert ((out[rest].double() - good[rest].double()).abs()
            <= 2.0**-7 * good[rest].double().abs() + 1e-3).all()
    assert not torch.isfinite(out[2]).all()
    m.moe_few_tokens(experts, c["x"], out, ws)
    assert torch.equal(out, good)


@pytest.mark.parametrize("bits", [4, 16])
def test_zero_tokens_and_tiny_ones(m, bits):
    c = make("flat", 3, BF16, bits, 32)
    experts = experts_of(m, c)
    ws = m.few_tokens_workspace(experts, 3)
    x, out = c["x"].clone(), torch.empty_like(c["x"])
    x[0] = 0
    x[1] = (x[1].float() * 2.0**-60).to(BF16)  # gate and up survive, h underflows to nothing
    m.moe_few_tokens(experts, x, out, ws)
    assert (out[0] == 0).all() and torch.isfinite(out).all() and float(out[1].abs().max()) < 1e-30
    assert m.moe_check_device_status(ws) == m.MOE_OK


@pytest.mark.parametrize("bits", [4, 16])
def test_the_same_bits_on_every_call_and_in_a_graph(m, bits):
    c = make("groups", 8, BF16, bits, 32)
    experts = experts_of(m, c)
    ws = m.few_tokens_workspace(experts, 8)
    out = torch.empty_like(c["x"])
    m.moe_few_tokens(experts, c["x"], out, ws)
    first = out.clone()
    for _ in range(20):
        out.fill_(7)
        m.moe_few_tokens(experts, c["x"], out, ws)
        assert torch.equal(out, first)
    graph = torch.cuda.CUDAGraph()
    x = c["x"].clone()
    with torch.cuda.graph(graph):
        m.moe_few_tokens(experts, x, out, ws)
        m.moe_few_tokens(experts, out, x, ws)  # back to back: the second reads the first's output
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first)
    again = torch.empty_like(x)
    m.moe_few_tokens(experts, first, again, ws)
    assert torch.equal(x, again)
    assert m.moe_check_device_status(ws) == m.MOE_OK


def test_one_workspace_for_batches_of_any_size(m):
    c = make("groups", 8, BF16, 4, 32)
    experts = experts_of(m, c)
    ws = m.few_tokens_workspace(experts, 8)
    want = torch.empty_like(c["x"])
    m.moe_few_tokens(experts, c["x"], want, ws)
    for T in (1, 8, 3, 2, 7):
        out = torch.empty_like(c["x"][:T])
        m.moe_few_tokens(experts, c["x"][:T], out, ws)
        assert ((out.double() - want[:T].double()).abs()
                <= 2.0**-7 * want[:T].double().abs() + 1e-3).all()
    m.moe_few_tokens(experts, c["x"][:0], c["x"][:0], ws)  # no tokens: nothing to do
    small = m.few_tokens_workspace(experts, 1)
    with pytest.raises(m.MoeError, match="workspace too small"):
        m.moe_few_tokens(experts, c["x"], want, small)


def test_two_streams_at_once(m):
    c = [make("deep", T, BF16, 4, 128, seed=T) for T in (1, 4)]
    experts = [experts_of(m, v) for v in c]
    streams = [torch.cuda.Stream() for _ in c]
    ws = [m.few_tokens_workspace(e, v["spec"]["T"]) for e, v in zip(experts, c)]
    want = [torch.empty_like(v["x"]) for v in c]
    outs = [torch.empty_like(v["x"]) for v in c]
    for e, v, w, o in zip(experts, c, ws, want):
        m.moe_few_tokens(e, v["x"], o, w)
    torch.cuda.synchronize()
    for _ in range(30):
        for e, v, w, o, s in zip(experts, c, ws, outs, streams):
            m.moe_few_tokens(e, v["x"], o, w, stream=s)
    torch.cuda.synchronize()
    for o, w, v in zip(outs, ws, want):
        assert torch.equal(o, v)
        assert m.moe_check_device_status(w) == m.MOE_OK


def test_launches_and_arguments(m):
    c = make("flat", 4, BF16, 16)
    experts = experts_of(m, c)
    ws = m.few_tokens_workspace(experts, 4)
    out = torch.empty_like(c["x"])
    before = m.launch_counts()
    m.moe_few_tokens(experts, c["x"], out, ws)
    after = m.launch_counts()
    assert {k: after[k] - before[k] for k in after if after[k] != before[k]} == \
        {"few_route": 1, "few_ffn": 1}
    for bad, error in ((dict(x=c["x"].half()), TypeError), (dict(x=c["x"][:, :256]), ValueError),
                       (dict(out=out.half()), TypeError), (dict(out=out[:2]), ValueError),
                       (dict(ws=None), TypeError), (dict(x=c["x"].cpu()), ValueError),
                       (dict(topk_ids=torch.empty(4, 4, device="cuda")), TypeError),
                       (dict(topk_w=torch.empty(4, 3, device="cuda")), ValueError)):
        a = dict(dict(x=c["x"], out=out, ws=ws), **bad)
        with pytest.raises(error):
            m.moe_few_tokens(experts, **a)
    with pytest.raises(m.MoeError, match="unsupported"):
        nine = torch.zeros(9, 512, dtype=BF16, device="cuda")
        m.moe_few_tokens(experts, nine, torch.empty_like(nine), ws)
    with pytest.raises(ValueError, match="requires a gradient"):
        m.moe_few_tokens(experts, c["x"], torch.empty_like(c["x"]).requires_grad_(), ws)


def test_as_the_layer_itself(m):
    """The same weights through moe_layer_forward, within both calls' roundings."""
    c = make("groups", 8, BF16, 16)
    got = check(m, c)
    spec, w = c["spec"], c["w"]
    cfg = m.config_from_spec(spec)
    out = torch.empty_like(got)
    ws = m.workspace(cfg, 8)
    m.moe_layer_forward(cfg, 8, c["x"], c["w_r"].cuda(), None, w["w_gate"], w["w_up"], w["w_down"],
                        None, None, None, w["shared_gate"], w["shared_up"], w["shared_down"], out,
                        ws)
    torch.cuda.synchronize()
    assert float((out.double() - got.double()).norm() / got.double().norm()) <= gs.REL_L2


def test_plain_launches_give_the_same_bits(m, tmp_path):
    """MOE_PDL=0 in another process: the second kernel then starts after the first."""
    code = (
        "import sys, torch\n"
        "from tests import test_gpu_few_tokens as t, gpu_support as gs\n"
        "m = gs.lib()\n"
        "c = t.make('groups', 8, torch.bfloat16, 4, 32)\n"
        "e = t.experts_of(m, c)\n"
        "o = torch.empty_like(c['x'])\n"
        "m.moe_few_tokens(e, c['x'], o, m.few_tokens_workspace(e, 8))\n"
        "torch.save(o.cpu(), sys.argv[1])\n")
    outs = []
    for pdl in ("0", "1"):
        at = str(tmp_path / pdl)
        subprocess.run([sys.executable, "-c", code, at], check=True, cwd=ROOT,
                       env=dict(os.environ, MOE_PDL=pdl), timeout=300)
        outs.append(torch.load(at))
    assert torch.equal(*outs)


@pytest.mark.parametrize("dtype,bits", [(BF16, 16), (FP16, 16), (BF16, 4)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_weights_that_are_not_finite_reach_their_tokens_only(m, dtype, bits, bad):
    c = make("deep", 6, dtype, bits, 64)
    experts = experts_of(m, c)
    ws = m.few_tokens_workspace(experts, 6)
    good, out = torch.empty_like(c["x"]), torch.empty_like(c["x"])
    ids = torch.empty(6, 4, dtype=torch.int32, device="cuda")
    m.moe_few_tokens(experts, c["x"], good, ws, ids)
    e = int(ids[2, 1])
    picked = (ids == e).any(1)
    assert picked.any() and not picked.all()
    for key in ("w_gate", "w_down") if bits == 16 else ("s_gate", "s_down"):
        c["w"][key][e].fill_(bad)
    m.moe_few_tokens(experts, c["x"], out, ws)
    torch.cuda.synchronize()
    assert torch.equal(out[~picked], good[~picked])
    assert not torch.isfinite(out[picked]).any()


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("T", [1, 4])
@pytest.mark.parametrize("name", ["flat", "deep"])
def test_an_infinite_h_gives_infinities(m, name, T, dtype):
    c = make(name, T, dtype, 16)
    c["x"][0, 0] = 0.5  # its gate becomes +inf: silu is infinite, not NaN
    spec = c["spec"]
    experts = experts_of(m, c)
    ws = m.few_tokens_workspace(experts, T)
    out = torch.empty_like(c["x"])
    ids = torch.empty(T, spec["top_k"], dtype=torch.int32, device="cuda")
    w = torch.empty(T, spec["top_k"], device="cuda")
    c["w"]["w_gate"][:, 3, 0] = float("inf")
    m.moe_few_tokens(experts, c["x"], out, ws, ids, w)
    torch.cuda.synchronize()
    e = int(ids[0, 0])
    # one expert alone: of two, infinities could cancel
    c["w"]["w_gate"][:, 3, 0] = 0.0
    c["w"]["w_gate"][e, 3, 0] = float("inf")
    m.moe_few_tokens(experts, c["x"], out, ws)
    torch.cuda.synchronize()
    up = c["w"]["w_up"][e, 3].double() @ c["x"][0].double()
    want = torch.sign(up) * c["w"]["w_down"][e, :, 3].double() * float("inf")
    assert torch.isinf(want).sum() > spec["hidden"] * 0.9
    got = out[0].double()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got[torch.isinf(want)], want[torch.isinf(want)])
    rest = [t for t in range(1, T) if e not in ids[t].tolist()]
    assert torch.isfinite(out[rest]).all()
    assert m.moe_check_device_status(ws) == m.MOE_OK


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("H,I,T", [(65536, 64, 1), (8192, 64, 8), (1024, 1 << 18, 8)])
def test_long_sums_are_rounded_on_the_way(m, H, I, T, dtype):
    """All terms positive, so that MMAs all cut off in one direction and relative errors add up.

    An output is the rounding of a number within d of the value.  Sixteen MMAs lose at most 17 u
    of their sum (2 u each of what is held then, 16 + 15 + .. + 1 of 16 parts); n such sums added,
    rounded, n / 2 + 1 u; the parts of four warps (gate and up) or sixteen (down) 4 or 16 u.  h
    has gate's (times 1.1, for silu') and up's, 16 u of its own, and its split, 2^-17 or 2^-22.
    A sixteenth more covers parts that are not alike.  A chain of K / 64 MMAs and more would lose
    hundreds of u, a good part of which shows in fp16's step, 8192 u."""
    spec = synth.spec("tiny", T=T, name="few_long", n_zero=0, renormalize=True, hidden=H, inter=I,
                      n_routed=1, top_k=1)
    g = gen(H + I)
    x = 0.5 + torch.rand(T, H, generator=g, device="cuda")
    # (gate's weights, about 24 / H: silu(24) is 24)
    w = {"w_gate": 0.5 + torch.rand(1, I, H, generator=g, device="cuda"),
         "w_up": 0.5 + torch.rand(1, I, H, generator=g, device="cuda"),
         "w_down": 0.5 + torch.rand(1, H, I, generator=g, device="cuda")}
    for key, scale in (("w_gate", 24 / H), ("w_up", 2 / H), ("w_down", 1 / I)):
        w[key] = w[key].mul_(scale).mul_(64 if dtype == FP16 and key == "w_down" else 1).to(dtype)
    x = x.to(dtype)
    experts = m.FewTokenExperts(m.config_from_spec(spec), w, torch.ones(1, H, device="cuda"))
    ws = m.few_tokens_workspace(experts, T)
    out = torch.empty_like(x)
    m.moe_few_tokens(experts, x, out, ws)
    torch.cuda.synchronize()
    assert m.moe_check_device_status(ws) == m.MOE_OK
    xd = x.double()

    def product(v, key):  # in parts: 64-bit copies of the large weights are too large
        return torch.cat([v @ part.double().T for part in w[key][0].split(1 << 14)], 1)

    gate, up = product(xd, "w_gate"), product(xd, "w_up")
    want = product(gate * torch.sigmoid(gate) * up, "w_down")
    assert float(want.min()) > 2.0**-10 and float(want.max()) < 2.0**15
    product_of = 17 + H / 256 / 4 / 2 + 1 + 4
    d = 2.1 * product_of + 16 + 17 + I / 64 / 16 / 2 / 2 + 1 + 16
    d = 17 / 16 * d * U + (2.0**-17 if dtype == BF16 else 2.0**-22)
    low, high = (want * (1 - d)).to(dtype), (want * (1 + d)).to(dtype)
    assert (out >= low).all() and (out <= high).all(), float(((out.double() - want) / want).abs().max())


def cut_product(w, key, infix, mat, e, v, dv=None):
    """A 4-bit matrix in groups of 32 times v (off by dv) in 64 bits, and the bound of its error.

    A block is four MMAs (two of codes, two of ones for the sum of v), each of sixteen products and
    what it starts from, cut off at 2^-15 of the largest |v|: 68 of that times the block's scale.
    Blocks, warps and scales are added and applied in fp32: 15 u of the magnitudes."""
    a, b = exact_matrix(w, key, infix, mat, e)
    s = w[f"s_{infix}{mat}"]
    s = (s if e is None else s[e]).double()
    top = (v.abs() + (0 if dv is None else dv)).max()
    tol = 15 * U * (b @ v.abs()) + 68 * 2.0**-15 * top * s.abs().sum(1) + \
        2.0**-33 * top * a.abs().sum(1)
    return a @ v, tol if dv is None else tol + a.abs() @ dv


def hidden_of(c, prefix, infix, e, x):
    """(h, bound of its error as the down projection takes it) of one expert for one token."""
    (g, dg), (u, du) = (cut_product(c["w"], prefix + mat, infix, mat, e, x) for mat in ("gate", "up"))
    silu = g * torch.sigmoid(g)
    h = silu * u
    dh = 1.1 * dg * u.abs() + (silu.abs() + 1.1 * dg) * du + 16 * U * h.abs()
    # one fp16 number where x is bf16 (half a step: eps / 2 = 2^-11), else two; 2^-34 of the largest
    rel = 2.0**-11 if c["dtype"] == BF16 else 2.0**-22
    return h, dh + rel * (h.abs() + dh) + 2.0**-34 * (h.abs() + dh).max()


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("T,E,k,Is", [(1, 1, 1, 0), (3, 2, 1, 64), (4, 8, 3, 0), (5, 1, 1, 64),
                                      (6, 3, 2, 32), (8, 1, 1, 0), (8, 2, 2, 96), (8, 16, 4, 64)])
@pytest.mark.parametrize("I", [64, 2080])
def test_differences_of_h_in_four_bit_layers(m, T, E, k, Is, I, dtype):
    """Rows of the down projection with +1 and -1 at two h of a token that are next to each other in
    size, for experts with one to eight tokens."""
    H = 96
    spec = synth.spec("tiny", T=T, name="few_h", n_zero=0, renormalize=True, hidden=H, inter=I,
                      n_routed=E, top_k=k, shared_inter=Is)
    g = gen(T + E + I)
    x = torch.randn(T, H, generator=g, device="cuda").to(BF16)
    x = torch.where(x.abs() < 2.0**-9, torch.zeros_like(x), x).to(dtype)
    c = dict(spec=spec, x=x, dtype=dtype, bits=4, w={})
    parts = [("w_", "", (E,), I)] + ([("shared_", "shared_", (), Is)] if Is else [])
    for prefix, infix, lead, inter in parts:
        for mat, n, kk in (("gate", inter, H), ("up", inter, H), ("down", H, inter)):
            c["w"][prefix + mat] = m.pack_w4(torch.randint(
                0, 16, (*lead, n, kk), generator=g, device="cuda", dtype=torch.uint8))
            c["w"][f"s_{infix}{mat}"] = (0.3 + torch.rand(*lead, n, kk // 32, generator=g,
                                                          device="cuda")) / (4.6 * H**0.5)
            c["w"][f"z_{infix}{mat}"] = torch.full((*lead, n, kk // 32), 8 if mat != "down" else 1,
                                                   dtype=torch.uint8, device="cuda")
        # down: zero points 1, codes 1 but for 2 and 0 at two neighbours in size among the larger h of
        # token row % T; scales 1 for their groups, 0 for the others
        q = torch.ones((*lead, H, inter), dtype=torch.uint8, device="cuda")
        s = torch.zeros((*lead, H, inter // 32), device="cuda")
        for e in range(E) if lead else (None,):
            qe, se = (q, s) if e is None else (q[e], s[e])
            for t in range(T):
                h = hidden_of(c, prefix, infix, e, x[t].double())[0]
                order = torch.argsort(h.abs(), descending=True)[:inter // 2]
                order = order[torch.argsort(h[order])]
                gaps = torch.argsort((h[order][1:] - h[order][:-1]).abs())
                for i, row in enumerate(range(t, H, T)):
                    j = int(gaps[i % (len(gaps) // 2)])
                    for at, code in ((int(order[j]), 2), (int(order[j + 1]), 0)):
                        qe[row, at], se[row, at // 32] = code, 1.0
        c["w"][prefix + "down"], c["w"][f"s_{infix}down"] = m.pack_w4(q), s
    w_r = torch.randn(E, H, generator=g, device="cuda")
    experts = m.FewTokenExperts(m.config_from_spec(spec), c["w"], w_r)
    ws = m.few_tokens_workspace(experts, T)
    out = torch.empty_like(x)
    ids = torch.empty(T, k, dtype=torch.int32, device="cuda")
    w = torch.empty(T, k, device="cuda")
    m.moe_few_tokens(experts, x, out, ws, ids, w)
    torch.cuda.synchronize()
    assert m.moe_check_device_status(ws) == m.MOE_OK
    for t in range(T):
        picks = [("w_", "", int(e), float(p)) for e, p in zip(ids[t], w[t])] + \
            ([("shared_", "shared_", None, 1.0)] if Is else [])
        want, tol = (torch.zeros(H, dtype=torch.float64, device="cuda") for _ in range(2))
        for prefix, infix, e, p in picks:
            y, dy = cut_product(c["w"], prefix + "down", infix, "down", e,
                                *hidden_of(c, prefix, infix, e, x[t].double()))
            want += p * y
            tol += p * (dy + 30 * U * y.abs())  # sixteen warps, picks, weights
        tol = tol + torch.finfo(dtype).eps / 2 * (want.abs() + tol) + TINY[dtype]
        over = ((out[t].double() - want).abs() - tol).max()
        assert float(over) <= 0, (t, float(over), float(tol.median()))


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("T,E,k,Is", [(1, 1, 1, 0), (2, 3, 2, 0), (3, 2, 1, 64), (4, 8, 3, 0),
                                      (5, 1, 1, 64), (6, 3, 2, 32), (7, 4, 4, 0), (8, 1, 1, 0),
                                      (8, 2, 2, 96), (8, 16, 4, 64)])
@pytest.mark.parametrize("I,group", [(64, 32), (2080, 32), (128, 64), (2304, 128)])
def test_h_of_fp16_layers_has_two_terms(m, T, E, k, Is, I, group, zeros, dtype):
    """The differences of neighbours again, of h that the MMAs add exactly: all between an eighth of
    the largest and it, so that their 11-bit terms are multiples of what an MMA cuts off at.

    x has one channel, so that gate and up are a code and a scale: exact but for fp32's roundings,
    16 u of h with silu's.  What is left is h's own rounding, half a step of fp16, eps / 2 = 2^-11 of
    it, with one term, 2^-22 with two, and 8 u of the magnitudes (q + z) h of its blocks, which z times their sum and the scales
    round to."""
    if group > 32:
        Is = up_to(Is, group)
    H = 128
    spec = synth.spec("tiny", T=T, name="few_h", n_zero=0, renormalize=True, hidden=H, inter=I,
                      n_routed=E, top_k=k, shared_inter=Is)
    g = gen(T + E + I)
    x = torch.zeros(T, H, device="cuda", dtype=dtype)
    x[:, 0] = 1 + torch.randperm(64, generator=g, device="cuda")[:T] / 128
    w, hs = {}, {}
    parts = [("w_", "", (E,), I)] + ([("shared_", "shared_", (), Is)] if Is else [])
    for prefix, infix, lead, inter in parts:
        for mat, n, kk in (("gate", inter, H), ("up", inter, H), ("down", H, inter)):
            q = torch.randint(0, 16, (*lead, n, kk), generator=g, device="cuda", dtype=torch.uint8)
            q[..., 0] = 9
            w[prefix + mat] = m.pack_w4(q)
            w[f"s_{infix}{mat}"] = 1 + torch.rand(*lead, n, kk // group, generator=g, device="cuda")
            if zeros:
                w[f"z_{infix}{mat}"] = torch.full((*lead, n, kk // group), 8, dtype=torch.uint8,
                                                  device="cuda")
        gate, up = (w[f"s_{infix}{mat}"][..., 0].double() for mat in ("gate", "up"))
        q = torch.full((*lead, H, inter), 8, dtype=torch.uint8, device="cuda")
        s = torch.zeros((*lead, H, inter // group), device="cuda")
        for e in range(E) if lead else (None,):
            qe, se = (q, s) if e is None else (q[e], s[e])
            for t in range(T):
                v = gate if e is None else gate[e]
                v = v * x[t, 0].double()
                h = v * torch.sigmoid(v) * (up if e is None else up[e]) * x[t, 0].double()
                assert float(h.min()) >= float(h.max()) / 8
                hs[e, t] = h
                order = torch.argsort(h)
                for i, row in enumerate(range(t, H, T)):
                    j = (37 * i + 11) % (inter - 1)
                    for at, code in ((int(order[j]), 9), (int(order[j + 1]), 7)):
                        qe[row, at], se[row, at // group] = code, 1.0
        w[prefix + "down"], w[f"s_{infix}down"] = m.pack_w4(q), s
    w_r = torch.randn(E, H, generator=g, device="cuda")
    experts = m.FewTokenExperts(m.config_from_spec(spec), w, w_r)
    ws = m.few_tokens_workspace(experts, T)
    out = torch.empty_like(x)
    ids = torch.empty(T, k, dtype=torch.int32, device="cuda")
    wts = torch.empty(T, k, device="cuda")
    m.moe_few_tokens(experts, x, out, ws, ids, wts)
    torch.cuda.synchronize()
    assert m.moe_check_device_status(ws) == m.MOE_OK
    rel = 16 * U + (2.0**-11 if dtype == BF16 else 2.0**-22)
    for t in range(T):
        picks = [("w_", "", int(e), float(p)) for e, p in zip(ids[t], wts[t])] + \
            ([("shared_", "shared_", None, 1.0)] if Is else [])
        want, tol = (torch.zeros(H, dtype=torch.float64, device="cuda") for _ in range(2))
        for prefix, infix, e, p in picks:
            a, b = exact_matrix(w, prefix + "down", infix, "down", e)
            h = hs[e, t]
            want += p * (a @ h)
            tol += p * ((rel + 30 * U) * (a.abs() @ h) + 8 * U * (b @ h))
        tol = tol + torch.finfo(dtype).eps / 2 * (want.abs() + tol) + TINY[dtype]
        over = ((out[t].double() - want).abs() - tol).max()
        assert float(over) <= 0, (t, float(over), float(tol.median()))


def up_to(v, to):
    return -(-v // to) * to


@pytest.mark.parametrize("T", [3, 8])
def test_paired_columns_stay_apart(m, T):
    """fp16 and 4-bit weights: tokens and experts that are not finite reach their own tokens only, and
    calls give the same bits, in a graph too."""
    c = make("deep", T, FP16, 4, 64, seed=3)
    k = c["spec"]["top_k"]
    experts = experts_of(m, c)
    ws = m.few_tokens_workspace(experts, T)
    good, out = torch.empty_like(c["x"]), torch.empty_like(c["x"])
    ids = torch.empty(T, k, dtype=torch.int32, device="cuda")
    m.moe_few_tokens(experts, c["x"], good, ws, ids)
    for _ in range(10):
        m.moe_few_tokens(experts, c["x"], out.fill_(7), ws)
        assert torch.equal(out, good)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.moe_few_tokens(experts, c["x"], out, ws)
    out.fill_(7)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, good)
    # a token
    for bad in (float("nan"), float("inf")):
        x = c["x"].clone()
        x[1, 5] = bad
        m.moe_few_tokens(experts, x, out, ws)
        rest = [t for t in range(T) if t != 1]
        assert torch.isfinite(out[rest]).all() and not torch.isfinite(out[1]).all()
        # (the other token's picks may differ, and with them the order of the sums)
        assert ((out[rest].double() - good[rest].double()).abs()
                <= 2.0**-10 * good[rest].double().abs() + 1e-4).all()
    # an expert
    e = int(ids[0, 0])
    picked = (ids == e).any(1)
    c["w"]["s_gate"][e].fill_(float("inf"))
    c["w"]["s_down"][e].fill_(float("inf"))
    m.moe_few_tokens(experts, c["x"], out, ws)
    torch.cuda.synchronize()
    assert torch.equal(out[~picked], good[~picked])
    assert not torch.isfinite(out[picked]).any()


@pytest.mark.parametrize("T", [1, 2, 5, 8])
@pytest.mark.parametrize("dtype,bits,zeros", [(BF16, 16, False), (FP16, 16, False), (BF16, 4, False),
                                              (FP16, 4, True)])
@pytest.mark.parametrize("inter", [50, 33, 4097])
def test_an_inter_that_no_expert_has(m, monkeypatch, inter, dtype, bits, zeros, T):
    # rows of h are the shared expert's, whole 16-byte pieces
    monkeypatch.setitem(LAYERS, "unused_inter", dict(hidden=256, inter=inter, n_routed=0, n_zero=4,
                                                     top_k=1, shared_inter=32))
    check(m, make("unused_inter", T, dtype, bits, 32, zeros, None))
