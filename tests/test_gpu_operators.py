"""The operators around the layer against their definitions in 64 bits.

Tolerances count roundings: u = 2^-24 for every fp32 operation on the way, plus
half a step of the output's type (eps / 2 relative, and half the smallest
subnormal where the type has few exponent bits).
"""
import numpy as np
import pytest
import torch

from tests import gpu_support as gs

pytestmark = pytest.mark.gpu

U = 2.0**-24
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
TINY = {BF16: 2.0**-134, FP16: 2.0**-25, FP32: 2.0**-150}


@pytest.fixture(scope="module")
def m():
    return gs.lib()


def gen(seed=0):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, dtype=FP32):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def strided(t, extra):
    """The same matrix with `extra` further channels between its rows, NaN there."""
    wide = torch.full((t.shape[0], t.shape[1] + extra), float("nan"), device=t.device).to(t.dtype)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


def within(got, want, tol, what=""):
    got, want = got.double(), want.double()
    assert torch.isfinite(got).all(), what
    over = (got - want).abs() - tol
    assert float(over.max()) <= 0, f"{what}: off by {float((got - want).abs().max()):.3e}, " \
        f"{float(over.max()):.3e} more than allowed"


def half_step(t, dtype):
    return torch.finfo(dtype).eps / 2 * t.abs() + TINY[dtype]


# ------------------------------------------------------------------ norm ----
# fp32 roundings of y: at most 4 * 8 squares a thread, 5 + 5 levels of the two
# reductions (halved by the square root), mean, eps, root, quotient, two
# products and the residual sum: below 32 u
NORM_REL = 32 * U


def norm_exact(x, res, gamma, eps):
    r = x.double() + (0 if res is None else res.double())
    v = r / torch.sqrt((r * r).mean(-1, keepdim=True) + eps)
    return r, v * (1 if gamma is None else gamma.double())


def check_norm(m, x, res, gamma, eps, qdt, group, extra=0):
    T, H = x.shape
    dt = x.dtype
    if extra:
        x, res = strided(x, extra), None if res is None else strided(res, extra)
    out = torch.full((T, H + extra), 7.0, device="cuda", dtype=dt)[:, :H]
    y = torch.full((T, H + 2 * extra), 7.0, device="cuda", dtype=dt)[:, :H]
    q = scale = None
    if qdt is not None:
        q = torch.zeros((T, H), device="cuda", dtype=torch.int8).view(qdt)
        scale = torch.full((T, -(-H // group) if group else 1), -1.0, device="cuda")
    m.moe_add_rmsnorm(x, res, gamma, eps, out, y, q, scale, group)
    torch.cuda.synchronize()
    r, want = norm_exact(x, res, gamma, eps)
    within(out, r, half_step(r, dt) + U * r.abs(), "sum")
    within(y, want, half_step(want, dt) + NORM_REL * want.abs(), "y")
    if q is None:
        return
    width = group or H
    G = scale.shape[1]
    pad = torch.nn.functional.pad(want, (0, G * width - H)).view(T, G, width)
    most = 127.0 if qdt == torch.int8 else 448.0
    s = pad.abs().amax(-1) / most
    within(scale, s, (NORM_REL + U) * s, "scale")
    code = q.to(FP32).double() if qdt != torch.int8 else q.double()
    value = torch.nn.functional.pad(code, (0, G * width - H)).view(T, G, width) \
        * scale.double()[..., None]
    rel = 2 * NORM_REL + 4 * U
    if qdt == torch.int8:
        assert int(q.to(torch.int32).abs().max()) <= 127
        tol = 0.5 * s[..., None] * (1 + rel) + rel * pad.abs()
    else:  # half a step: 2^-4 relative, or half of e4m3's smallest subnormal 2^-9
        tol = (2.0**-4 + rel) * pad.abs() + 2.0**-10 * s[..., None] * (1 + rel)
    within(value, pad, tol, "codes")


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("T,H", [(1, 1), (1, 7), (2, 8), (1, 7168), (5, 1000), (3, 1024), (7, 250),
                                 (33, 5120), (2, 8200), (1, 16392), (2, 32768), (3, 32761)])
def test_norm_shapes(m, dtype, T, H):
    g = gen(T * 100000 + H)
    x, res = randn(g, T, H, dtype=dtype), 3 * randn(g, T, H, dtype=dtype)
    gamma = (1 + 0.2 * randn(g, H)).to(dtype)
    for qdt, group in ((None, 0), (torch.int8, 0), (torch.float8_e4m3fn, 128)):
        check_norm(m, x, res, gamma, 1e-6, qdt, group)


@pytest.mark.parametrize("T", [400, 1999])
@pytest.mark.parametrize("H", [96, 1000, 1001, 1024, 2048, 7168, 16384])
def test_norm_many_rows(m, T, H):
    # several rows a CTA: the reductions of consecutive rows must not mix
    g = gen(H + T)
    x, res = randn(g, T, H, dtype=BF16), randn(g, T, H, dtype=BF16)
    x *= torch.exp(3 * randn(g, T, 1)).to(BF16)  # rows of very different size
    check_norm(m, x, res, (1 + 0.2 * randn(g, H)).to(BF16), 1e-5, torch.int8, 0)


@pytest.mark.parametrize("qdt", [torch.int8, torch.float8_e4m3fn])
@pytest.mark.parametrize("group", [0, 32, 64, 128, 256])
@pytest.mark.parametrize("H", [40, 1000, 4104, 777])
def test_norm_codes(m, qdt, group, H):
    g = gen(group + H)
    x = randn(g, 9, H, dtype=FP16)
    x[:, 3] *= 50  # a loud channel sets its group's scale alone
    check_norm(m, x, None, None, 1e-6, qdt, group)


@pytest.mark.parametrize("extra", [8, 3])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_norm_row_strides(m, extra, dtype):
    g = gen(extra)
    check_norm(m, randn(g, 6, 512, dtype=dtype), randn(g, 6, 512, dtype=dtype),
               randn(g, 512, dtype=dtype), 1e-6, torch.int8, 64, extra)


def test_norm_in_place(m):
    g = gen(5)
    x, res = randn(g, 300, 2048, dtype=BF16), randn(g, 300, 2048, dtype=BF16)
    a, b = torch.empty_like(x), torch.empty_like(x)
    m.moe_add_rmsnorm(x, res, None, 1e-6, a, b)
    m.moe_add_rmsnorm(x, res, None, 1e-6, res, x)  # the residual is updated, y replaces x
    assert torch.equal(res, a) and torch.equal(x, b)


def test_norm_zero_rows_and_tiny_rows(m):
    x = torch.zeros(4, 256, device="cuda", dtype=FP32)
    x[1] = 1e-30
    x[2] = 2.0**-140  # subnormal: codes must not overflow on the way
    x[3, 5] = 1.0
    q = torch.ones(4, 256, dtype=torch.int8, device="cuda")
    s = torch.ones(4, 1, device="cuda")
    gamma = torch.full((256,), 1e-12, device="cuda")
    m.moe_add_rmsnorm(x, None, gamma, 1e-6, None, None, q, s)
    torch.cuda.synchronize()
    assert int(q[0].abs().max()) == 0 and float(s[0]) == 0.0
    assert (q[1] == 127).all() and torch.isfinite(s).all()
    assert (q[3] == torch.eye(256, dtype=torch.int8, device="cuda")[5] * 127).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_norm_rows_that_are_not_finite_stay_apart(m, bad):
    g = gen(1)
    x = randn(g, 5, 512, dtype=BF16)
    x[2, 77] = bad
    y, q = torch.empty_like(x), torch.empty(5, 512, dtype=torch.int8, device="cuda")
    s = torch.empty(5, 1, device="cuda")
    m.moe_add_rmsnorm(x, None, None, 1e-6, None, y, q, s)
    torch.cuda.synchronize()
    rest = [0, 1, 3, 4]
    assert torch.isfinite(y[rest]).all() and torch.isfinite(s[rest]).all()
    assert torch.isnan(s[2]).all() and torch.isnan(y[2, 77])
    if bad != bad:
        assert torch.isnan(y[2]).all()
    else:
        assert (y[2, :77] == 0).all()


def test_norm_codes_of_whole_numbers(m):
    # the codes do not depend on the row's norm: round(r * 127 / 128), exactly
    x = torch.arange(-128, 128, device="cuda").to(BF16).repeat(3, 1)
    rms = float(torch.sqrt((x.double() ** 2).mean(-1))[0])
    q, s = torch.empty(3, 256, dtype=torch.int8, device="cuda"), torch.empty(3, 1, device="cuda")
    m.moe_add_rmsnorm(x, None, None, 0.0, None, None, q, s)
    torch.cuda.synchronize()
    want = torch.round(x.double() * 127 / 128)
    assert torch.equal(q.double(), want)
    assert abs(float(s[0]) * rms * 127 / 128 - 1) < 64 * U


# ---------------------------------------------------------- sort and back ----
def plan_exact(ids, E):
    key = ids.cpu().numpy().reshape(-1).astype(np.int64)
    key = np.where((key >= 0) & (key < E), key, E)
    order = np.argsort(key, kind="stable")
    inverse = np.empty_like(order)
    inverse[order] = np.arange(len(order))
    counts = np.bincount(key, minlength=E + 1)[:E]
    return order, inverse, counts, np.concatenate([[0], np.cumsum(counts)])


def run_sort(m, ids, E, x, x_scale=None, zero_dropped=True, fill=7):
    T, k = ids.shape
    i32 = dict(dtype=torch.int32, device="cuda")
    p = dict(counts=torch.full((E,), -5, **i32), offsets=torch.full((E + 1,), -5, **i32),
             s2e=torch.full((T * k,), -5, **i32), e2s=torch.full((T * k,), -5, **i32))
    xs = ss = None
    if x is not None:
        xs = torch.full((T * k, x.shape[1]), fill, device="cuda", dtype=FP32).to(x.dtype)
    if x_scale is not None:
        ss = torch.full((T * k,), 7.0, device="cuda")
    m.moe_sort_tokens(E, ids, x, x_scale, p["counts"], p["offsets"], p["s2e"], p["e2s"], xs, ss,
                      m.sort_workspace(T, k, E), zero_dropped)
    torch.cuda.synchronize()
    return p, xs, ss


def draw_ids(g, T, k, E, over=0, distinct=True):
    if distinct:
        return torch.argsort(torch.rand(T, E + over, generator=g, device="cuda"))[:, :k].int() \
            .contiguous()
    return torch.randint(-2, E + 2, (T, k), generator=g, device="cuda", dtype=torch.int32)


def check_sort(m, ids, E, x, zero_dropped=True, scale=None):
    p, xs, ss = run_sort(m, ids, E, x, scale, zero_dropped)
    order, inverse, counts, offsets = plan_exact(ids, E)
    assert np.array_equal(p["s2e"].cpu().numpy(), order)
    assert np.array_equal(p["e2s"].cpu().numpy(), inverse)
    assert np.array_equal(p["counts"].cpu().numpy(), counts)
    assert np.array_equal(p["offsets"].cpu().numpy(), offsets)
    if x is None:
        return
    n, k = int(offsets[-1]), ids.shape[1]
    src = torch.from_numpy(order // k).cuda()
    bits = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[x.element_size()]
    got, row = xs.view(bits), x.contiguous().view(bits)
    assert torch.equal(got[:n], row[src[:n]])
    rest = xs[n:].to(FP32)
    assert (rest == (0 if zero_dropped else 7)).all()
    if scale is not None:
        assert torch.equal(ss[:n], scale[src[:n]])
        assert (ss[n:] == (0 if zero_dropped else 7)).all()


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 256), (2, 3, 5), (64, 12, 512), (33, 32, 64),
                                   (512, 8, 64), (513, 8, 64), (1000, 7, 100), (4096, 2, 8),
                                   (3001, 5, 160), (300, 32, 4096), (70000, 1, 16), (9000, 1, 1)])
@pytest.mark.parametrize("kind", ["distinct", "dropped", "repeated"])
def test_sort_orders(m, T, k, E, kind):
    g = gen(T + k + E)
    over = E // 2 if kind == "dropped" else 0
    if kind == "distinct" and k > E:
        pytest.skip("more picks than experts")
    ids = draw_ids(g, T, min(k, E + over) if kind != "repeated" else k, E, over,
                   kind != "repeated")
    check_sort(m, ids, E, randn(g, T, 24, dtype=BF16))


@pytest.mark.parametrize("T,k", [(1, 4), (40, 4), (3000, 2)])
@pytest.mark.parametrize("value", [-1, 16, 0, 15, 2**31 - 1, -(2**31)])
def test_sort_all_picks_alike(m, T, k, value):
    ids = torch.full((T, k), value, dtype=torch.int32, device="cuda")
    check_sort(m, ids, 16, randn(gen(3), T, 40, dtype=FP16))


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32, torch.int8, torch.float8_e4m3fn])
@pytest.mark.parametrize("H", [1, 3, 6, 20, 72, 1000, 1001, 6144])
@pytest.mark.parametrize("T", [50, 1100])
def test_sort_rows(m, dtype, H, T):
    g = gen(H + T)
    x = (20 * randn(g, T, H)).to(dtype)
    ids = draw_ids(g, T, 4, 16, 8)
    check_sort(m, ids, 16, x, scale=torch.rand(T, generator=g, device="cuda"))
    check_sort(m, ids, 16, x, zero_dropped=False,
               scale=torch.rand(T, 1, generator=g, device="cuda").view(T))


@pytest.mark.parametrize("extra", [1, 2, 8])
def test_sort_row_strides(m, extra):
    g = gen(extra)
    for T in (30, 2500):
        x = torch.randn(T, 256 + extra, generator=g, device="cuda").to(BF16)[:, :256]
        check_sort(m, draw_ids(g, T, 2, 12), 12, x)


def test_sort_order_only(m):
    g = gen(9)
    for T in (10, 5000):
        check_sort(m, draw_ids(g, T, 4, 32, 4), 32, None)


def test_sort_agrees_with_the_layers_re_sort(m):
    import synth

    spec = synth.spec("dsv3_s")
    g = gen(2)
    T, k, E, H = spec["T"], spec["top_k"], spec["n_routed"], spec["hidden"]
    ids, x = draw_ids(g, T, k, E), randn(g, T, H, dtype=BF16)
    cfg = m.config_from_spec(spec)
    i32 = dict(dtype=torch.int32, device="cuda")
    counts, offsets = torch.empty(E, **i32), torch.empty(E + 1, **i32)
    s2e, e2s = torch.empty(T * k, **i32), torch.empty(T * k, **i32)
    xp = torch.empty(T * k, H, dtype=BF16, device="cuda")
    m.moe_permute(cfg, T, ids, x, counts, offsets, s2e, e2s, xp, None, m.workspace(cfg, T))
    p, xs, _ = run_sort(m, ids, E, x)
    assert torch.equal(p["s2e"], s2e) and torch.equal(p["e2s"], e2s)
    assert torch.equal(p["counts"], counts) and torch.equal(p["offsets"], offsets)
    assert torch.equal(xs, xp)


def test_sort_offsets_past_32_bits(m):
    # 2.2e9 elements, 4.3e9 bytes of sorted rows
    g = gen(4)
    T, H = 66000, 32776
    x = torch.randint(-99, 100, (T, H), generator=g, device="cuda", dtype=torch.int8).view(
        torch.int8)
    ids = torch.randint(0, 3, (T, 2), generator=g, device="cuda", dtype=torch.int32)
    p, xs, _ = run_sort(m, ids, 3, x)
    src = p["s2e"].long() // 2
    for a in range(0, 2 * T, 11000):
        assert torch.equal(xs[a:a + 11000], x[src[a:a + 11000]])
    del xs, x
    y = torch.randn(T * 2, 1, generator=g, device="cuda").to(BF16).expand(-1, H).contiguous()
    w = torch.rand(T, 2, generator=g, device="cuda")
    out = torch.empty(T, H, device="cuda", dtype=BF16)
    m.moe_unsort_tokens(y, p["offsets"], p["e2s"], w, out)
    torch.cuda.synchronize()
    want = (y[:, 0].double()[p["e2s"].long()].view(T, 2) * w.double()).sum(1)
    for col in (0, H - 1):
        within(out[:, col], want, half_step(want, BF16) + 1e-6)


def back_case(g, T, k, E, H, dtype, out_dtype, over=0):
    ids = draw_ids(g, T, k, E, over)
    order, inverse, counts, offsets = plan_exact(ids, E)
    t = dict(y=randn(g, T * k, H, dtype=dtype), dout=randn(g, T, H, dtype=out_dtype),
             w=torch.rand(T, k, generator=g, device="cuda"),
             e2s=torch.from_numpy(inverse).int().cuda(),
             offsets=torch.from_numpy(offsets).int().cuda())
    kept = int(offsets[-1])
    t["y"][kept:] = float("nan")  # rows of dropped picks are never read
    at = t["e2s"].long().view(T, k)
    t["mask"] = (at < kept)
    rows = torch.where(t["mask"].reshape(-1, 1), t["y"].double()[at.reshape(-1)], 0.0).view(T, k, H)
    return t, rows, at, kept


BACK = [(1, 1, 1, 8, 0), (1, 8, 64, 7168, 0), (3, 2, 4, 1, 0), (37, 5, 16, 1000, 8),
        (200, 4, 8, 333, 3), (700, 8, 32, 256, 16), (2, 32, 40, 2100, 24), (310, 3, 6, 4104, 0)]


@pytest.mark.parametrize("T,k,E,H,over", BACK)
@pytest.mark.parametrize("dtype,out_dtype", [(BF16, BF16), (BF16, FP32), (FP16, FP16), (FP32, FP32),
                                             (FP32, BF16), (FP16, FP32), (FP32, FP16)])
def test_unsort_and_gradients(m, T, k, E, H, over, dtype, out_dtype):
    g = gen(T + H)
    t, rows, at, kept = back_case(g, T, k, E, H, dtype, out_dtype, over)
    w, R = t["w"].double(), T * k
    out = torch.full((T, H), 7.0, device="cuda", dtype=out_dtype)
    m.moe_unsort_tokens(t["y"], t["offsets"], t["e2s"], t["w"], out)
    dx = torch.full((T, H), 7.0, device="cuda", dtype=out_dtype)
    m.moe_sort_tokens_backward(t["y"], t["offsets"], t["e2s"], k, dx)
    dy = torch.full((R, H), 7.0, device="cuda", dtype=dtype)
    dw = torch.full((T, k), 7.0, device="cuda")
    m.moe_unsort_tokens_backward(t["dout"], t["y"], t["offsets"], t["e2s"], t["w"], dy, dw)
    torch.cuda.synchronize()
    # k products and additions in fp32, then one rounding
    terms = w[..., None] * rows
    want = terms.sum(1)
    within(out, want, half_step(want, out_dtype) * (1 + 2 * k * U) + 2 * k * U * terms.abs().sum(1),
           "out")
    want = rows.sum(1)
    within(dx, want, half_step(want, out_dtype) * (1 + 2 * k * U) + k * U * rows.abs().sum(1), "dx")
    d = t["dout"].double()
    want = torch.where(t["mask"][..., None], w[..., None] * d[:, None, :], 0.0)
    want_sorted = torch.zeros(R, H, dtype=torch.float64, device="cuda")
    want_sorted[at.reshape(-1)] = want.view(R, H)
    within(dy, want_sorted, half_step(want_sorted, dtype) + U * want_sorted.abs(), "dy")
    prod = rows * d[:, None, :]
    # a thread adds 8 products a segment of 2048 channels, a warp 32 lanes in 5
    # levels, then segments and 8 warps one after another
    seg = -(-H // 2048)
    within(dw, prod.sum(-1), (8 + 5 + seg + 8 + 1) * U * prod.abs().sum(-1), "dw")
    assert (dw[~t["mask"]] == 0).all()


def test_unsort_backward_leaves_dropped_rows_alone_when_asked(m):
    t, _, _, kept = back_case(gen(8), 50, 4, 8, 64, BF16, BF16, 8)
    dy = torch.full((200, 64), 7.0, device="cuda", dtype=BF16)
    dw = torch.empty(50, 4, device="cuda")
    m.moe_unsort_tokens_backward(t["dout"], t["y"], t["offsets"], t["e2s"], t["w"], dy, dw,
                                 zero_dropped=False)
    torch.cuda.synchronize()
    assert kept < 200 and (dy[kept:] == 7).all() and (dw[~t["mask"]] == 0).all()


@pytest.mark.parametrize("extra", [3, 8])
def test_unsort_row_strides(m, extra):
    T, k, H = 60, 2, 128
    t, rows, at, _ = back_case(gen(extra), T, k, 8, H, BF16, BF16)
    out = torch.empty(T, H + extra, device="cuda", dtype=BF16)
    m.moe_unsort_tokens(t["y"], t["offsets"], t["e2s"], t["w"], out[:, :H])
    flat = torch.empty(T, H, device="cuda", dtype=BF16)
    m.moe_unsort_tokens(t["y"], t["offsets"], t["e2s"], t["w"], flat)
    assert torch.equal(out[:, :H], flat)
    got = [torch.empty_like(t["y"]) for _ in range(2)], [torch.empty(T, k, device="cuda")
                                                         for _ in range(2)]
    for i, d in enumerate((t["dout"], strided(t["dout"], extra))):
        m.moe_unsort_tokens_backward(d, t["y"], t["offsets"], t["e2s"], t["w"], got[0][i],
                                     got[1][i])
    torch.cuda.synchronize()
    assert torch.equal(*got[0]) and torch.equal(*got[1])


def test_gradients_against_differences(m):
    # out is linear in y and in w, so central differences of L = <G, out> of any
    # width are exact but for the roundings of the two forward passes
    T, k, E, H = 40, 4, 8, 200
    g = gen(11)
    t, _, at, kept = back_case(g, T, k, E, H, FP32, FP32, 4)
    t["y"][kept:] = 0
    G = t["dout"]
    dy, dw = torch.empty_like(t["y"]), torch.empty_like(t["w"])
    m.moe_unsort_tokens_backward(G, t["y"], t["offsets"], t["e2s"], t["w"], dy, dw)

    def loss(y, w):
        out = torch.empty(T, H, device="cuda")
        m.moe_unsort_tokens(y, t["offsets"], t["e2s"], w, out)
        return float((out.double() * G.double()).sum())

    def bound(y, w):  # 2k roundings a value of out, and as many of the gradient's own
        rows = y.abs().double()[at.reshape(-1)].view(T, k, H)
        return float(((w.abs().double()[..., None] * rows).sum(1) * G.abs().double()).sum()) \
            * (4 * k + 30) * U

    uy, uw = randn(g, *t["y"].shape), randn(g, T, k)
    uy[kept:] = 0
    for y2, w2, grad in (((t["y"] + uy, t["y"] - uy), (t["w"], t["w"]), (dy.double() * uy).sum()),
                         ((t["y"], t["y"]), (t["w"] + uw, t["w"] - uw), (dw.double() * uw).sum())):
        diff = (loss(y2[0], w2[0]) - loss(y2[1], w2[1])) / 2
        tol = bound(y2[0], w2[0]) + bound(y2[1], w2[1])
        assert abs(diff - float(grad)) <= tol, (diff, float(grad), tol)
    # dx of the sorted rows: L = <D, sort(x)> is linear in x
    ids = draw_ids(g, T, k, E, 4)
    x, ux = randn(g, T, H), randn(g, T, H)
    p, xs, _ = run_sort(m, ids, E, x)
    _, us, _ = run_sort(m, ids, E, ux)
    D = randn(g, T * k, H)
    dx = torch.empty(T, H, device="cuda")
    m.moe_sort_tokens_backward(D, p["offsets"], p["e2s"], k, dx)
    want = float((D.double() * us.double()).sum())
    tol = float((D.abs().double() * us.abs().double()).sum()) * 2 * k * U
    assert abs(float((dx.double() * ux.double()).sum()) - want) <= tol


def test_positions_outside_the_rows_are_skipped(m):
    # a plan that is not this batch's: nothing outside the tensors is touched
    T, k, H = 20, 2, 64
    g = gen(6)
    y, w = randn(g, T * k, H, dtype=BF16), torch.rand(T, k, generator=g, device="cuda")
    offsets = torch.tensor([0, 10**9], dtype=torch.int32, device="cuda")
    e2s = torch.full((T * k,), 10**6, dtype=torch.int32, device="cuda")
    e2s[1::2] = -3
    out = torch.full((T, H), 7.0, device="cuda", dtype=BF16)
    m.moe_unsort_tokens(y, offsets, e2s, w, out)
    dy, dw = torch.full_like(y, 7.0), torch.full_like(w, 7.0)
    m.moe_unsort_tokens_backward(out, y, offsets, e2s, w, dy, dw)
    torch.cuda.synchronize()
    assert (out == 0).all() and (dw == 0).all() and (dy == 7).all()


# ------------------------------------------------- streams, graphs, launches --
def test_side_stream_and_graph_replay(m):
    T, k, E, H = 24, 4, 16, 512
    g = gen(7)
    x, res = randn(g, T, H, dtype=BF16), randn(g, T, H, dtype=BF16)
    ids, w = draw_ids(g, T, k, E), torch.rand(T, k, generator=g, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    y, out = torch.empty_like(x), torch.empty_like(x)
    counts, offsets = torch.empty(E, **i32), torch.empty(E + 1, **i32)
    s2e, e2s = torch.empty(T * k, **i32), torch.empty(T * k, **i32)
    xs = torch.empty(T * k, H, dtype=BF16, device="cuda")
    dy, dw, dx = torch.empty_like(xs), torch.empty_like(w), torch.empty_like(x)

    def step(stream=None):
        m.moe_add_rmsnorm(x, res, None, 1e-6, None, y, stream=stream)
        m.moe_sort_tokens(E, ids, y, None, counts, offsets, s2e, e2s, xs, stream=stream)
        m.moe_unsort_tokens(xs, offsets, e2s, w, out, stream=stream)
        m.moe_unsort_tokens_backward(out, xs, offsets, e2s, w, dy, dw, stream=stream)
        m.moe_sort_tokens_backward(dy, offsets, e2s, k, dx, stream=stream)

    results = (y, counts, offsets, s2e, e2s, xs, out, dy, dw, dx)
    step()
    torch.cuda.synchronize()
    want = [r.clone() for r in results]
    side = torch.cuda.Stream()
    for r in results:
        r.zero_()
    torch.cuda.synchronize()
    step(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(results, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    x2 = randn(g, T, H, dtype=BF16)
    x.copy_(x2)
    step()
    torch.cuda.synchronize()
    want = [r.clone() for r in results]
    for r in results:
        r.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(results, want))


# ---------------------------------------------------------------- 4 bits ----
INT8 = torch.int8


def w4_case(g, E, R, N, K, group, xdt, sdt, up, zeros, rows=None):
    G = K // group if group else 1
    t = dict(up=up, group=group or K)
    t["x_scale"] = None
    if xdt == INT8:
        t["x"] = torch.randint(-127, 128, (R, K), generator=g, device="cuda", dtype=INT8)
        t["x_scale"] = 0.01 + torch.rand(R, generator=g, device="cuda")
    else:
        t["x"] = randn(g, R, K, dtype=xdt)
    for n in ("", "_up")[:2 if up else 1]:
        t["codes" + n] = torch.randint(0, 16, (E, N, K), generator=g, device="cuda",
                                       dtype=torch.uint8)
        t["scales" + n] = ((0.5 + torch.rand(E, N, G, generator=g, device="cuda")) / K**0.5).to(sdt)
        t["zeros" + n] = torch.randint(0, 17, (E, N, G), generator=g, device="cuda",
                                       dtype=torch.uint8) if zeros else None
    if rows is None:
        cut = torch.sort(torch.randint(0, R + 1, (E - 1,), generator=g, device="cuda")).values
        rows = [0] + cut.tolist() + [R]
    t["bounds"] = rows
    t["offsets"] = torch.tensor(rows, dtype=torch.int32, device="cuda")
    return t


def w4_exact(t, e, n=""):
    q = t["codes" + n][e].double()
    z = t["zeros" + n]
    q = q - (8 if z is None else z[e].double().repeat_interleave(t["group"], 1))
    q = q * t["scales" + n][e].double().repeat_interleave(t["group"], 1)
    a, b = t["bounds"][e], t["bounds"][e + 1]
    x = t["x"][a:b].double()
    if t["x_scale"] is not None:
        x = x * t["x_scale"][a:b, None].double()
    return x @ q.T, x.abs() @ q.abs().T


def run_w4(m, t, out_dtype, offsets="given", fill=7.0):
    R, N = t["x"].shape[0], t["codes"].shape[1]
    out = torch.full((R, N), fill, device="cuda", dtype=out_dtype)
    up = [None] * 3
    if t["up"]:
        up = [m.pack_w4(t["codes_up"]), t["scales_up"], t["zeros_up"]]
    m.moe_w4_gemv(t["x"], t["x_scale"], t["offsets"] if offsets == "given" else offsets,
                  m.pack_w4(t["codes"]), t["scales"], t["zeros"], out, *up)
    torch.cuda.synchronize()
    return out


def check_w4(m, t, out_dtype, offsets="given"):
    out = run_w4(m, t, out_dtype, offsets)
    K = t["x"].shape[1]
    # products are exact; a sum of at most 128 of them is 8 MMA steps that may
    # each lose a step of 2^-23 per term, then one fp32 addition a group, the K
    # parts, the scales and the row scale
    rel = (8 * 17 + K // 32 + 20) * 2.0**-23
    for e in range(len(t["bounds"]) - 1):
        a, b = t["bounds"][e], t["bounds"][e + 1]
        if a == b:
            continue
        y, mag = w4_exact(t, e)
        tol = rel * mag
        if t["up"]:
            u, umag = w4_exact(t, e, "_up")
            silu = y * torch.sigmoid(y)
            # |d silu / dy| <= 1.1
            tol = 1.1 * tol * (u.abs() + rel * umag) + silu.abs() * rel * umag \
                + 8 * U * (silu * u).abs()
            y = silu * u
        within(out[a:b], y, half_step(y, out_dtype) * (1 + rel) + tol, f"expert {e}")
    covered = t["bounds"][-1]
    assert (out[covered:] == 7).all()


@pytest.mark.parametrize("xdt", [BF16, FP16, INT8])
@pytest.mark.parametrize("group", [32, 64, 128, 0])
@pytest.mark.parametrize("up,zeros", [(False, False), (True, False), (False, True), (True, True)])
def test_w4_types_and_groups(m, xdt, group, up, zeros):
    g = gen(group + 2 * up + zeros)
    t = w4_case(g, 3, 21, 200, 640, group, xdt, FP32 if xdt == INT8 else xdt, up, zeros)
    check_w4(m, t, FP32)
    check_w4(m, t, BF16)


@pytest.mark.parametrize("E,R,N,K,group", [
    (1, 1, 1, 32, 32), (1, 1, 16, 64, 64), (1, 8, 127, 96, 0), (1, 9, 129, 160, 32),
    (1, 16, 64, 2048, 128), (1, 17, 65, 2080, 32), (1, 40, 130, 1056, 0), (1, 1, 7168, 2048, 128),
    (1, 3, 33, 16384, 128), (1, 2, 500, 7200, 32), (4, 5, 256, 512, 64), (16, 37, 1000, 1024, 32),
    (64, 9, 96, 256, 128), (2, 100, 300, 544, 32), (5, 64, 72, 4096, 64)])
@pytest.mark.parametrize("xdt,up", [(BF16, False), (INT8, True)])
def test_w4_shapes(m, E, R, N, K, group, xdt, up):
    g = gen(E + R + N + K)
    check_w4(m, w4_case(g, E, R, N, K, group, xdt, BF16, up, False), FP32)


@pytest.mark.parametrize("sdt", [BF16, FP16, FP32])
@pytest.mark.parametrize("out_dtype", [BF16, FP16, FP32])
def test_w4_scale_and_output_types(m, sdt, out_dtype):
    check_w4(m, w4_case(gen(1), 2, 12, 136, 384, 128, FP16, sdt, True, True), out_dtype)


@pytest.mark.parametrize("rows", [[0, 0, 0, 5, 5], [0, 5, 5, 5, 5], [0, 1, 2, 3, 4],
                                  [0, 0, 40, 40, 41], [0, 0, 0, 0, 0], [0, 8, 16, 24, 30]])
def test_w4_loads(m, rows):
    # empty experts, one expert with everything, rows that no expert owns
    check_w4(m, w4_case(gen(3), 4, 41, 150, 256, 64, BF16, BF16, False, False, rows), BF16)


def test_w4_one_expert_without_offsets(m):
    t = w4_case(gen(4), 1, 6, 100, 512, 32, FP16, FP16, True, False)
    check_w4(m, t, FP32, offsets=None)


def test_w4_offsets_that_are_not_a_plan_stay_inside(m):
    t = w4_case(gen(5), 3, 10, 64, 128, 32, BF16, BF16, False, False)
    bad = torch.tensor([-5, 4, 10**9, 2], dtype=torch.int32, device="cuda")
    run_w4(m, t, BF16, bad)  # rows 0-3, 4-9 and none: nothing outside is touched
    out = run_w4(m, t, BF16, torch.full((4,), 99, dtype=torch.int32, device="cuda"))
    assert (out == 7).all()


def test_w4_rows_do_not_mix(m):
    t = w4_case(gen(6), 2, 11, 96, 256, 64, BF16, BF16, False, False, [0, 7, 11])
    clean = run_w4(m, t, FP32)
    t["x"][2, 5] = float("nan")
    t["x"][9, 0] = float("inf")
    got = run_w4(m, t, FP32)
    rest = [r for r in range(11) if r not in (2, 9)]
    assert torch.equal(got[rest], clean[rest])
    assert torch.isnan(got[2]).all() and not torch.isfinite(got[9]).all()


def test_w4_same_bits_every_call_and_graph_replay(m):
    t = w4_case(gen(7), 8, 24, 512, 2048, 128, BF16, BF16, True, False)
    first = run_w4(m, t, FP32)
    for _ in range(3):
        assert torch.equal(run_w4(m, t, FP32), first)
    w, wu = m.pack_w4(t["codes"]), m.pack_w4(t["codes_up"])
    out = torch.zeros_like(first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.moe_w4_gemv(t["x"], None, t["offsets"], w, t["scales"], None, out, wu, t["scales_up"])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first)


def test_w4_weights_past_32_bits(m):
    # 2.4e9 bytes of codes: the last experts lie beyond 2^31
    E, N, K = 320, 2048, 7168
    g = gen(8)
    w = torch.randint(0, 256, (E, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = torch.full((E, N, 1), 0.01, device="cuda", dtype=BF16)
    x = randn(g, 2, K, dtype=BF16)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[E - 1:] = torch.tensor([1, 2], dtype=torch.int32)
    out = torch.empty(2, N, device="cuda")
    m.moe_w4_gemv(x, None, off, w, s, None, out)
    torch.cuda.synchronize()
    for r, e in ((0, E - 2), (1, E - 1)):
        q = torch.stack([w[e] & 15, w[e] >> 4], -1).view(N, K).double() - 8
        q *= float(s[0, 0, 0])
        rel = (8 * 17 + K // 32 + 20) * 2.0**-23
        within(out[r], q @ x[r].double(), rel * (q.abs() @ x[r].abs().double()) + TINY[FP32])


# ----------------------------------------------------- together, as used ----
def test_autograd_functions_against_torch(m):
    from sparse_expert_layer_gb300 import autograd

    T, k, E, H = 50, 3, 8, 120
    g = gen(12)
    ids = draw_ids(g, T, k, E, 3)
    x, w, c = randn(g, T, H), torch.rand(T, k, generator=g, device="cuda"), randn(g, T * k, H)
    grad_out = randn(g, H, T).T  # not contiguous: taken as a copy

    def plain(x, w, c):
        order, inverse, _, offsets = plan_exact(ids, E)
        src = torch.from_numpy(order // k).cuda()
        kept = (torch.arange(T * k, device="cuda") < int(offsets[-1]))[:, None]
        xs = x[src] * kept
        y = torch.tanh(xs) * c
        rows = (y * kept)[torch.from_numpy(inverse).cuda()].view(T, k, H)
        return (rows * w[..., None]).sum(1)

    a = [t.clone().requires_grad_() for t in (x, w, c)]
    xs, plan = autograd.sort_tokens(a[0], ids, E)
    out = autograd.unsort_tokens(torch.tanh(xs) * a[2], a[1], plan)
    out.backward(grad_out)
    b = [t.double().requires_grad_() for t in (x, w, c)]
    want = plain(*b)
    want.backward(grad_out.double())
    # sums of a few products near 1 in size (dw: 120 of them), fp32 throughout
    out, want = out.detach(), want.detach()
    assert torch.allclose(out.double(), want, rtol=0, atol=64 * U * float(want.abs().max()))
    for p, q in zip(a, b):
        assert torch.allclose(p.grad.double(), q.grad, rtol=0,
                              atol=256 * U * float(q.grad.abs().max()))


def test_example_block_against_64_bits(m):
    import importlib.util
    import os

    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "w4_block.py")
    spec = importlib.util.spec_from_file_location("w4_block", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    us, block, x, start, residual = ex.decode()
    assert us > 0
    T, H = x.shape
    r, y = norm_exact(x, start, block.gamma, 1e-6)
    within(residual, r, half_step(r, BF16) + U * r.abs(), "residual")
    within(block.y, y, half_step(y, BF16) + NORM_REL * y.abs(), "y")
    # from the codes and the routing on, every step is checked on its inputs
    xq = block.q.double() * block.q_scale.double()
    assert float((xq - y).abs().max()) <= 0.51 * float(block.q_scale.max())

    def dequant(packed, scales):
        q = torch.stack([packed & 15, packed >> 4], -1).view(*packed.shape[:2], -1).double() - 8
        return q * scales.double().repeat_interleave(q.shape[2] // scales.shape[2], 2)

    wg, wu, wd = (dequant(*p) for p in (block.gate, block.up, block.down))
    want = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    size = torch.zeros_like(want)
    for j in range(block.k):
        e = block.ids[:, j].long()
        gate = torch.einsum("th,tih->ti", xq, wg[e])
        h = gate * torch.sigmoid(gate) * torch.einsum("th,tih->ti", xq, wu[e])
        w = block.weights[:, j, None].double()
        want += w * torch.einsum("ti,thi->th", h, wd[e])
        size += w * torch.einsum("ti,thi->th", h.abs(), wd[e].abs())
    # h is rounded to bf16 between the products, the output once more
    within(block.out, want, half_step(want, BF16) + (2.0**-8) * size, "block output")
    losses = ex.train()
    assert losses[-1] < 0.9 * losses[0]


def test_empty_batches_on_the_device(m):
    i32 = dict(dtype=torch.int32, device="cuda")
    x = torch.empty(0, 64, device="cuda", dtype=BF16)
    m.moe_add_rmsnorm(x, None, None, 1e-6, x.clone())
    ids = torch.empty(0, 2, **i32)
    p, xs, _ = run_sort(m, ids, 5, x)
    assert (p["counts"] == 0).all() and (p["offsets"] == 0).all() and xs.shape == (0, 64)
    m.moe_unsort_tokens(xs, p["offsets"], p["e2s"], torch.empty(0, 2, device="cuda"), x)
    out = torch.empty(0, 8, device="cuda")
    m.moe_w4_gemv(x, None, torch.zeros(3, **i32), torch.zeros(2, 8, 32, dtype=torch.uint8,
                                                              device="cuda"),
                  torch.ones(2, 8, 1, device="cuda"), None, out)
    torch.cuda.synchronize()


def test_refused_sizes_raise_and_leave_the_context_usable(m):
    x = torch.zeros(4, 64, device="cuda", dtype=BF16)
    with pytest.raises(m.MoeError, match="misaligned"):
        m.moe_add_rmsnorm(torch.zeros(300, device="cuda", dtype=BF16)[4:260].view(4, 64), None, None,
                          1e-6, x)
    with pytest.raises(ValueError, match="shape"):
        m.moe_add_rmsnorm(x, x[:2], None, 1e-6, x)
    with pytest.raises(ValueError, match="not on CUDA device"):
        m.moe_add_rmsnorm(x, x.cpu(), None, 1e-6, x)
    with pytest.raises(TypeError, match="gamma"):
        m.moe_add_rmsnorm(x, None, torch.ones(64, device="cuda"), 1e-6, x)
    ids = torch.zeros(9000, 4, dtype=torch.int32, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    plan = (torch.empty(8, **i32), torch.empty(9, **i32), torch.empty(36000, **i32),
            torch.empty(36000, **i32))
    with pytest.raises(m.MoeError, match="invalid"):
        m.moe_sort_tokens(8, ids, None, None, *plan, None)  # no workspace
    m.moe_add_rmsnorm(x, None, None, 1e-6, x)
    torch.cuda.synchronize()


def test_launches_are_counted(m):
    before = m.launch_counts()
    x = torch.zeros(4, 64, device="cuda", dtype=BF16)
    m.moe_add_rmsnorm(x, None, None, 1e-6, x)
    run_sort(m, torch.zeros(4, 2, dtype=torch.int32, device="cuda"), 4, x)
    after = m.launch_counts()
    assert after["norm"] == before["norm"] + 1
    assert after["sort_rows"] == before["sort_rows"] + 1
    assert after["sort_plan"] == before["sort_plan"]
