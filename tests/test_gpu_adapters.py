"""moe_adapters and moe_adapters_backward against their definitions in 64 bits, and the
gradients against differences.

Tolerance, element by element, u = 2^-24: a sum of n products leaves at most
(n / 8 + 64) u times the sum of the magnitudes added (an MMA of sixteen products rounds
within two u of what it holds; blocks, warps and a cluster's parts follow).  v and u then
enter the next product as two 16-bit numbers, 2^-17 of them lost in bf16 and 2^-22 in
fp16, or in the sums over positions as three bf16 (2^-24) or two fp16 numbers (2^-22, and
2^-36 of the adapter's largest).  What is stored is rounded once.
"""
import pytest
import torch

from tests import gpu_support as gs

pytestmark = pytest.mark.gpu

U = 2.0**-24
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
TINY = {BF16: 2.0**-134, FP16: 2.0**-25, FP32: 2.0**-150}
SPLIT = {BF16: 2.0**-17, FP16: 2.0**-22}


@pytest.fixture(scope="module")
def m():
    return gs.lib()


def gen(seed=0):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, dtype=FP32):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def make(T, J, r, K, N, dtype, none=0.2, seed=0, ids=None):
    g = gen(seed + T + K)
    if ids is None:
        ids = torch.randint(0, J, (T,), generator=g, device="cuda")
        ids = torch.where(torch.rand(T, generator=g, device="cuda") < none, J, ids)
    c = dict(T=T, J=J, r=r, K=K, N=N, dtype=dtype, ids=ids)
    c["order"] = torch.sort(ids, stable=True).indices.int()
    c["offsets"] = (ids[None, :] < torch.arange(J + 1, device="cuda")[:, None]).sum(1).int()
    c["x"], c["base"] = randn(g, T, K, dtype=dtype), randn(g, T, N, dtype=dtype)
    c["dy"] = randn(g, T, N, dtype=dtype)
    c["a"] = (randn(g, J, r, K) / K**0.5).to(dtype)
    c["b"] = (randn(g, J, r, N) / r**0.5).to(dtype)
    c["scale"] = 0.5 + torch.rand(J, generator=g, device="cuda")
    return c


def within(got, want, tol, what=""):
    got = got.double()
    assert torch.isfinite(got).all(), what
    over = (got - want).abs() - tol
    assert over.numel() == 0 or float(over.max()) <= 0, \
        f"{what}: off by {float((got - want).abs().max()):.3e}, {float(over.max()):.3e} too much"


def rounded(want, tol, dtype):
    return tol + torch.finfo(dtype).eps / 2 * (want.abs() + tol) + TINY[dtype]


def product(x, m, dx=None):
    """x @ m and the bound of its error; dx: that of x."""
    want, size = x @ m, x.abs() @ m.abs()
    tol = (x.shape[-1] / 8 + 64) * U * size
    return want, tol if dx is None else tol + dx @ m.abs()


def exact(c):
    """Everything in 64 bits, with bounds: v [T, r] by row, y, and the gradients."""
    f = {k: c[k].double() for k in ("x", "base", "dy", "a", "b", "scale")}
    T, J, r = c["T"], c["J"], c["r"]
    z = lambda *s: torch.zeros(*s, dtype=torch.float64, device="cuda")  # noqa: E731
    out = {k: [z(*s), z(*s)] for k, s in (
        ("v", (T, r)), ("y", (T, c["N"])), ("dx", (T, c["K"])), ("da", (J, r, c["K"])),
        ("db", (J, r, c["N"])))}
    out["y"][0] += f["base"]
    split = SPLIT[c["dtype"]]
    term = 2.0**-24 if c["dtype"] == BF16 else 2.0**-22
    rows = [torch.nonzero(c["ids"] == j)[:, 0] for j in range(J)]
    us = {}
    for j, t in enumerate(rows):
        if not len(t):
            continue
        s = f["scale"][j]
        v, dv = product(f["x"][t], f["a"][j].T)
        out["v"][0][t], out["v"][1][t] = v, dv
        d, dd = product(v, f["b"][j], dv + split * v.abs())
        out["y"][0][t] += s * d
        out["y"][1][t] = s * dd + 4 * U * (s * d.abs() + out["y"][0][t].abs())
        u, du = product(f["dy"][t], f["b"][j].T)
        u, du = s * u, s * du + 2 * U * s * u.abs()
        us[j] = u, du
        out["dx"][0][t], out["dx"][1][t] = product(u, f["a"][j], du + split * u.abs())
    for j, t in enumerate(rows):
        if not len(t):
            continue
        s = f["scale"][j]
        u, du = us[j]
        v, dv = out["v"][0][t], out["v"][1][t]
        top_u, top_v = float((u.abs() + du).max()), float((v.abs() + dv).max())
        out["da"][0][j], out["da"][1][j] = product(
            u.T, f["x"][t], (du + term * u.abs() + 2.0**-36 * top_u).T)
        g, dg = product(v.T, f["dy"][t], (dv + term * v.abs() + 2.0**-36 * top_v).T)
        out["db"][0][j], out["db"][1][j] = s * g, s * dg + 2 * U * s * g.abs()
    return out


def wide(t, extra, fill=float("nan")):
    w = torch.full((t.shape[0], t.shape[1] + extra), fill, dtype=t.dtype, device="cuda")
    w[:, :t.shape[1]] = t
    return w[:, :t.shape[1]]


def check(m, c, extra=0, backward=True, grad_dtype=FP32):
    T, J, r, K, N, dt = (c[k] for k in ("T", "J", "r", "K", "N", "dtype"))
    want = exact(c)
    ws = torch.full((m.moe_adapters_workspace_size(T, r, K, N) + 256,), 255, dtype=torch.uint8,
                    device="cuda")
    use = ws[:-256]
    x, base, dy = wide(c["x"], extra), wide(c["base"], extra), wide(c["dy"], extra)
    y = wide(torch.full_like(c["base"], 7), 2 * extra, 7)
    v = torch.full((T, r), 7.0, device="cuda")
    plan = c["offsets"], c["order"]
    m.moe_adapters(x, c["a"], c["b"], c["scale"], *plan, base, y, v, use)
    torch.cuda.synchronize()
    within(y, want["y"][0], rounded(*want["y"], dt), "y")
    kept = int(c["offsets"][-1])
    o = c["order"].long()[:kept]
    within(v[:kept], want["v"][0][o], want["v"][1][o], "v")
    assert (v[kept:] == 7).all()
    # in place, without v: the same bits, and rows without an adapter as they were
    m.moe_adapters(x, c["a"], c["b"], c["scale"], *plan, base, base, None, use)
    assert torch.equal(base, y)
    # no base
    m.moe_adapters(x, c["a"], c["b"], c["scale"], *plan, None, y, None, use)
    d, dd = want["y"][0] - c["base"].double(), want["y"][1]
    within(y, d, rounded(d, dd, dt), "without a base")
    if extra:
        assert (y.as_strided((T, 2 * extra), y.stride(), N) == 7).all()
    if not backward:
        return
    dx = wide(torch.full_like(c["x"], 7), extra, 7)
    da = torch.full((J, r, K), 7.0, device="cuda", dtype=grad_dtype)
    db = torch.full((J, r, N), 7.0, device="cuda", dtype=grad_dtype)
    args = dy, x, v, c["a"], c["b"], c["scale"], *plan
    m.moe_adapters_backward(*args, dx, da, db, use)
    torch.cuda.synchronize()
    within(dx, want["dx"][0], rounded(*want["dx"], dt), "dx")
    within(da, want["da"][0], rounded(*want["da"], grad_dtype), "da")
    within(db, want["db"][0], rounded(*want["db"], grad_dtype), "db")
    again = [torch.full_like(t, 3) for t in (dx, da, db)]
    m.moe_adapters_backward(*args, again[0], None, None, use)
    m.moe_adapters_backward(*args, None, again[1], again[2], use)
    for p, q in zip((dx, da, db), again):
        assert torch.equal(p, q)
    assert (ws[-256:] == 255).all()


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("T,J,r,K,N", [
    (1, 1, 1, 1, 1), (1, 3, 16, 5120, 1024), (2, 1, 8, 64, 40), (5, 8, 16, 1000, 2048),
    (64, 48, 16, 7168, 2048), (63, 5, 7, 100, 333), (64, 1, 128, 512, 264), (33, 40, 64, 2048, 96),
    (65, 3, 16, 1024, 512), (129, 2, 17, 72, 776), (200, 300, 16, 512, 512), (200, 4, 1, 256, 8),
    (130, 9, 33, 1001, 515), (333, 5, 24, 1000, 1544), (1000, 3, 64, 520, 1288),
    (700, 20, 128, 640, 256), (257, 1, 100, 128, 1032), (2100, 2, 16, 4096, 264),
])
def test_shapes(m, dtype, T, J, r, K, N):
    check(m, make(T, J, r, K, N, dtype))


@pytest.mark.parametrize("extra", [8, 3])
@pytest.mark.parametrize("T", [7, 150])
def test_row_strides(m, extra, T):
    check(m, make(T, 4, 16, 264, 520, BF16), extra)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("T", [30, 300])
def test_gradients_of_the_16_bit_type(m, dtype, T):
    check(m, make(T, 4, 16, 512, 264, dtype), grad_dtype=dtype)


@pytest.mark.parametrize("T", [40, 400])
@pytest.mark.parametrize("which", ["none", "one", "ends", "alternating", "all_of_the_last"])
def test_plans(m, T, which):
    J = 6
    ids = {"none": torch.full((T,), J), "one": torch.full((T,), 3),
           "ends": torch.where(torch.arange(T) < T - 1, 0, J - 1),
           "alternating": torch.arange(T) % (J + 1), "all_of_the_last": torch.full((T,), J - 1)}
    check(m, make(T, J, 16, 256, 128, BF16, ids=ids[which].cuda()))


@pytest.mark.parametrize("T", [50, 400])
def test_sorted_rows_need_no_order(m, T):
    ids = torch.sort(torch.randint(0, 5, (T,), generator=gen(T), device="cuda")).values
    c = make(T, 4, 16, 256, 264, BF16, ids=ids)
    y, z = torch.empty_like(c["base"]), torch.empty_like(c["base"])
    ws = m.adapters_workspace(T, 16, 256, 264)
    m.moe_adapters(c["x"], c["a"], c["b"], c["scale"], c["offsets"], c["order"], c["base"], y, None,
                   ws)
    m.moe_adapters(c["x"], c["a"], c["b"], c["scale"], c["offsets"], None, c["base"], z, None, ws)
    assert torch.equal(y, z)
    want = exact(c)
    within(z, want["y"][0], rounded(*want["y"], BF16), "y")


@pytest.mark.parametrize("T", [50, 400])
def test_plans_from_the_sort(m, T):
    from sparse_expert_layer_gb300 import autograd

    c = make(T, 7, 16, 256, 264, BF16)
    ids = torch.where(c["ids"] == 7, -1 if T == 50 else 999, c["ids"]).int()
    plan = autograd.plan_adapters(ids, 7)
    assert torch.equal(plan.offsets, c["offsets"])
    assert torch.equal(plan.sorted_to_expanded, c["order"])


@pytest.mark.parametrize("T", [20, 300])
def test_offsets_and_rows_out_of_range_are_skipped(m, T):
    c = make(T, 3, 16, 128, 128, BF16)
    y = torch.full_like(c["base"], 7)
    ws = m.adapters_workspace(T, 16, 128, 128)
    v = torch.zeros(T, 16, device="cuda")
    a = c["x"], c["a"], c["b"], None
    order = c["order"].clone()
    gone = order[::3].long()
    order[::3] = torch.tensor([-1, T, 2**31 - 1], device="cuda", dtype=torch.int32).repeat(T)[
        :len(order[::3])]
    m.moe_adapters(*a, c["offsets"], order, c["base"], y, v, ws)
    good = torch.empty_like(y)
    m.moe_adapters(*a, c["offsets"], c["order"], c["base"], good, None, ws)
    torch.cuda.synchronize()
    stay = torch.ones(T, dtype=torch.bool, device="cuda")
    stay[gone] = False
    assert (y[gone] == 7).all() and torch.equal(y[stay], good[stay])
    dx, da, db = torch.empty_like(c["x"]), torch.empty(3, 16, 128, device="cuda"), \
        torch.empty(3, 16, 128, device="cuda")
    m.moe_adapters_backward(c["dy"], c["x"], v, c["a"], c["b"], None, c["offsets"], order, dx, da,
                            db, ws)
    for offsets in ([0, T, T + 5, 2**31 - 1], [-9, -5, 3, 2], [5, 5, 5, 5], [T, 0, T, 0]):
        off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
        m.moe_adapters(*a, off, c["order"], c["base"], y, v, ws)
        m.moe_adapters_backward(c["dy"], c["x"], v, c["a"], c["b"], None, off, c["order"], dx, da,
                                db, ws)
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("T", [20, 300])
def test_loud_and_quiet_rows(m, dtype, T):
    # v and u pass fp16's range, and rows differ by many binades
    c = make(T, 3, 16, 512, 256, dtype)
    for k in ("x", "dy"):
        c[k] = (c[k].float() * torch.exp2(torch.randint(-9, 10, (T, 1), generator=gen(5),
                                                        device="cuda").float())).to(dtype)
    c["a"] = (c["a"].float() * 64).to(dtype)
    c["b"] = (c["b"].float() / 64).to(dtype)
    check(m, c)


@pytest.mark.parametrize("T", [20, 300])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_rows_that_are_not_finite_stay_alone(m, T, bad):
    c = make(T, 3, 16, 256, 128, BF16, none=0.0)
    ws = m.adapters_workspace(T, 16, 256, 128)
    good, y = torch.empty_like(c["base"]), torch.empty_like(c["base"])
    plan = c["scale"], c["offsets"], c["order"]
    m.moe_adapters(c["x"], c["a"], c["b"], *plan, c["base"], good, None, ws)
    c["x"][5, 7] = bad
    m.moe_adapters(c["x"], c["a"], c["b"], *plan, c["base"], y, None, ws)
    rest = torch.arange(T, device="cuda") != 5
    assert torch.equal(y[rest], good[rest]) and not torch.isfinite(y[5]).all()


@pytest.mark.parametrize("T", [40, 500])
def test_the_same_bits_on_every_call_and_in_a_graph(m, T):
    c = make(T, 5, 16, 1024, 512, BF16)
    ws = m.adapters_workspace(T, 16, 1024, 512)
    outs = [torch.empty_like(c["base"]), torch.empty(T, 16, device="cuda"), torch.empty_like(c["x"]),
            torch.empty(5, 16, 1024, device="cuda"), torch.empty(5, 16, 512, device="cuda")]
    outs[1].zero_()

    def step():
        m.moe_adapters(c["x"], c["a"], c["b"], c["scale"], c["offsets"], c["order"], c["base"],
                       outs[0], outs[1], ws)
        m.moe_adapters_backward(c["dy"], c["x"], outs[1], c["a"], c["b"], c["scale"], c["offsets"],
                                c["order"], *outs[2:], ws)

    step()
    first = [t.clone() for t in outs]
    for _ in range(5):
        step()
        assert all(torch.equal(p, q) for p, q in zip(outs, first))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in (0, 2, 3, 4):
        outs[i].fill_(7)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(outs, first))


def test_two_streams_at_once(m):
    sets = [make(T, 5, 16, 2048, 1024, BF16, seed=T) for T in (48, 900)]
    state = []
    for c in sets:
        T = c["T"]
        y = torch.empty_like(c["base"])
        ws = m.adapters_workspace(T, 16, 2048, 1024)
        a = (c["x"], c["a"], c["b"], c["scale"], c["offsets"], c["order"], c["base"], y, None, ws)
        m.moe_adapters(*a)
        state.append((a, y.clone(), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for a, _, s in state:
            m.moe_adapters(*a, stream=s)
    torch.cuda.synchronize()
    for a, want, _ in state:
        assert torch.equal(a[7], want)


def test_arguments(m):
    c = make(10, 3, 16, 64, 40, BF16)
    y, ws = torch.empty_like(c["base"]), m.adapters_workspace(10, 16, 64, 40)
    v = torch.zeros(10, 16, device="cuda")
    good = dict(x=c["x"], a=c["a"], b=c["b"], scale=c["scale"], offsets=c["offsets"],
                order=c["order"], base=c["base"], y=y, v=None, ws=ws)
    before = m.launch_counts()["adapters"]
    m.moe_adapters(**good)
    assert m.launch_counts()["adapters"] - before == 1
    for bad, error in ((dict(x=c["x"].float()), TypeError), (dict(a=c["a"].half()), TypeError),
                       (dict(a=c["a"][0]), TypeError), (dict(b=c["b"][:2]), ValueError),
                       (dict(x=c["x"][:, :32]), ValueError), (dict(y=y[:, :8]), ValueError),
                       (dict(base=c["base"][:5]), ValueError), (dict(ws=None), TypeError),
                       (dict(order=c["order"].long()), TypeError),
                       (dict(offsets=c["offsets"][:3]), ValueError),
                       (dict(scale=c["scale"].double()), TypeError), (dict(v=v[:, :3]), ValueError),
                       (dict(ws=ws[:256]), m.MoeError), (dict(x=c["x"].cpu()), ValueError),
                       (dict(y=y.clone().requires_grad_()), ValueError)):
        with pytest.raises(error):
            m.moe_adapters(**dict(good, **bad))
    dx, da, db = torch.empty_like(c["x"]), torch.empty(3, 16, 64, device="cuda"), \
        torch.empty(3, 16, 40, device="cuda")
    good = dict(dy=c["dy"], x=c["x"], v=v, a=c["a"], b=c["b"], scale=None, offsets=c["offsets"],
                order=None, dx=dx, da=da, db=db, ws=ws)
    m.moe_adapters_backward(**good)
    m.moe_adapters_backward(**dict(good, x=None, v=None, da=None, db=None))
    for bad, error in ((dict(da=None), ValueError), (dict(dx=None, da=None, db=None), ValueError),
                       (dict(x=None), TypeError), (dict(v=None), TypeError),
                       (dict(da=da.half()), TypeError), (dict(db=db.bfloat16()), TypeError),
                       (dict(dx=dx.float()), TypeError), (dict(dy=c["dy"][:, :8]), ValueError)):
        with pytest.raises(error):
            m.moe_adapters_backward(**dict(good, **bad))


def test_no_rows(m):
    c = make(0, 3, 16, 64, 40, BF16)
    ws = m.adapters_workspace(0, 16, 64, 40)
    y, v = torch.empty_like(c["base"]), torch.zeros(0, 16, device="cuda")
    m.moe_adapters(c["x"], c["a"], c["b"], None, c["offsets"], c["order"], None, y, v, ws)
    da, db = torch.ones(3, 16, 64, device="cuda"), torch.ones(3, 16, 40, device="cuda")
    m.moe_adapters_backward(c["dy"], c["x"], v, c["a"], c["b"], None, c["offsets"], c["order"], None,
                            da, db, ws)
    assert (da == 0).all() and (db == 0).all()


@pytest.mark.parametrize("T", [24, 200])
def test_gradients_against_differences(m, T):
    """Through autograd, along random directions, in 64-bit differences of the definition."""
    from sparse_expert_layer_gb300 import autograd

    c = make(T, 3, 8, 96, 64, BF16)
    plan = autograd.plan_adapters(c["ids"].int(), 3)
    leaves = [c[k].clone().requires_grad_() for k in ("base", "x", "a", "b")]
    y = autograd.adapters(leaves[0], leaves[1], leaves[2], leaves[3], c["scale"], plan)
    y.backward(c["dy"])
    has = (c["ids"] < 3)[:, None]
    pick = c["ids"].clamp(max=2)

    def loss(base, x, a, b):
        d = torch.einsum("tk,trk->tr", x, a[pick])
        d = torch.einsum("tr,trn->tn", d, b[pick]) * c["scale"].double()[pick][:, None]
        return ((base + torch.where(has, d, 0.0)) * c["dy"].double()).sum()

    at = [t.detach().double() for t in leaves]
    for i, leaf in enumerate(leaves):
        d = randn(gen(i), *leaf.shape).double()
        step = 1e-4
        up, dn = [list(at), list(at)]
        up[i], dn[i] = at[i] + step * d, at[i] - step * d
        want = (loss(*up) - loss(*dn)) / (2 * step)
        got = (leaf.grad.double() * d).sum()
        # each element of the gradient is rounded to bf16, by at most 2^-8 of it
        tol = 2.0**-8 * (leaf.grad.double() * d).abs().sum() + 1e-6 * abs(float(want))
        assert abs(float(got - want)) <= float(tol)


def test_autograd_of_parts_and_layouts(m):
    from sparse_expert_layer_gb300 import autograd

    c = make(100, 3, 8, 96, 64, BF16)
    plan = autograd.plan_adapters(c["ids"].int(), 3)
    full = [c[k].clone().requires_grad_() for k in ("x", "a", "b")]
    autograd.adapters(c["base"], *full, None, plan).backward(c["dy"])
    # a frozen input, weights of another layout, a gradient that is expanded
    x = c["x"].t().contiguous().t()
    a = c["a"].transpose(0, 1).contiguous().transpose(0, 1).requires_grad_()
    y = autograd.adapters(None, x, a, c["b"], None, plan)
    y.backward(c["dy"])
    assert torch.equal(a.grad, full[1].grad)
    x = c["x"].clone().requires_grad_()
    autograd.adapters(None, x, c["a"], c["b"], None, plan).sum().backward()
    ones = c["x"].clone().requires_grad_()
    autograd.adapters(None, ones, c["a"], c["b"], None, plan).backward(torch.ones_like(c["dy"]))
    assert torch.equal(x.grad, ones.grad)
    with pytest.raises(RuntimeError, match="once_differentiable|not require grad"):
        y = autograd.adapters(None, ones, c["a"], c["b"], None, plan)
        (g,) = torch.autograd.grad(y.sum(), ones, create_graph=True)
        g.sum().backward()


@pytest.mark.parametrize("T", [24, 200])
def test_evaluation_with_a_scale_that_is_a_parameter(m, T):
    from sparse_expert_layer_gb300 import autograd

    c = make(T, 3, 8, 96, 64, BF16)
    plan = autograd.plan_adapters(c["ids"].int(), 3)
    args = c["base"], c["x"], c["a"], c["b"]
    want = autograd.adapters(*args, c["scale"], plan)
    scale = torch.nn.Parameter(c["scale"].clone())
    with torch.no_grad():
        assert torch.equal(autograd.adapters(*args, scale, plan), want)
    with pytest.raises(RuntimeError, match="scale"):
        autograd.adapters(*args, scale, plan)


@pytest.mark.parametrize("T", [24, 200])
def test_a_slice_of_a_scale(m, T):
    from sparse_expert_layer_gb300 import autograd

    c = make(T, 3, 8, 96, 64, BF16)
    plan = autograd.plan_adapters(c["ids"].int(), 3)
    scales = torch.cat([torch.full((1,), 9.0, device="cuda"), c["scale"]])
    got = []
    for scale in (c["scale"], scales[1:]):
        leaves = [c[k].clone().requires_grad_() for k in ("x", "a", "b")]
        y = autograd.adapters(c["base"], *leaves, scale, plan)
        y.backward(c["dy"])
        got.append([y.detach()] + [t.grad for t in leaves])
    assert all(torch.equal(p, q) for p, q in zip(*got))


def test_a_training_step_in_a_graph(m):
    """Forward, backward and clipping captured while eager gradients of the same leaves live."""
    from sparse_expert_layer_gb300 import autograd

    c = make(200, 3, 16, 256, 128, BF16)
    plan = autograd.plan_adapters(c["ids"].int(), 3)
    leaves = [c[k].clone().requires_grad_() for k in ("a", "b")]
    ws, norm = m.clip_workspace(), torch.zeros(1, device="cuda")
    x, w = c["x"], randn(gen(9), 128, 256, dtype=BF16) / 16
    grads = [torch.zeros_like(t) for t in leaves]

    def step():
        y = autograd.adapters(x @ w.T, x, *leaves, c["scale"], plan)
        got = torch.autograd.grad((y.float() ** 2).sum(), leaves)
        for g, n in zip(grads, got):
            g.copy_(n)
        m.moe_clip_grad_norm(grads, 1.0, norm, ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    first = [t.clone() for t in grads + [norm]]
    total = sum(float((t.double() ** 2).sum()) for t in grads) ** 0.5
    assert float(norm) > 1 and abs(total - 1) < 2.0**-7
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in grads + [norm]:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(grads + [norm], first))


# By rows the adapters are read from L2 again for every position; above 304 rows or 20 << 20 products
# T * r * (K + N) (8 << 20 above rank 16), and with more than two rows an adapter, positions go in tiles.
def tiled(r=16, K=1000, N=1016, J=5, T=None, **kw):
    T = T or (18 << 20) // (r * (K + N)) + 70
    assert T > 2 * J and (T > 304 or T * r * (K + N) > (20 << 20 if r <= 16 else 8 << 20))
    return make(T, J, r, K, N, kw.pop("dtype", BF16), **kw)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("r,K,N", [(1, 4000, 9), (15, 9, 3001), (16, 1003, 1001), (17, 1002, 1000),
                                   (32, 1001, 400), (33, 1000, 402), (64, 72, 1015), (65, 777, 8),
                                   (128, 1, 600), (127, 260, 255)])
def test_odd_sizes_in_tiles(m, dtype, r, K, N):
    check(m, tiled(r, K, N, dtype=dtype))


@pytest.mark.parametrize("extra", [8, 3])
@pytest.mark.parametrize("r", [16, 64])
def test_row_strides_in_tiles(m, extra, r):
    check(m, tiled(r), extra)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("r", [8, 48])
def test_gradients_of_the_16_bit_type_in_tiles(m, dtype, r):
    check(m, tiled(r, dtype=dtype), grad_dtype=dtype)


@pytest.mark.parametrize("r", [16, 128])
@pytest.mark.parametrize("which", ["none", "one", "ends", "alternating", "all_of_the_last", "sixty",
                                   "one_each"])
def test_plans_in_tiles(m, which, r):
    T = 700 if r == 16 else 160
    J = 64 if which == "one_each" else 6
    at = torch.arange(T)
    ids = {"none": torch.full((T,), J), "one": torch.full((T,), 3),
           "ends": torch.where(at < T - 1, 0, J - 1), "alternating": at % (J + 1),
           "all_of_the_last": torch.full((T,), J - 1),
           "sixty": torch.clamp(at // 64, max=J),  # whole tiles
           "one_each": torch.where(at < J, at, J)}[which]
    check(m, tiled(r, J=J, T=T, ids=ids.cuda()))


@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_loud_and_quiet_rows_in_tiles(m, dtype):
    c = tiled(dtype=dtype)
    for k in ("x", "dy"):
        c[k] = (c[k].float() * torch.exp2(torch.randint(-9, 10, (c["T"], 1), generator=gen(5),
                                                        device="cuda").float())).to(dtype)
    c["a"] = (c["a"].float() * 64).to(dtype)
    c["b"] = (c["b"].float() / 64).to(dtype)
    check(m, c)


def test_offsets_and_rows_out_of_range_are_skipped_in_tiles(m):
    c = tiled(J=3)
    T, r, K, N = (c[k] for k in ("T", "r", "K", "N"))
    ws = m.adapters_workspace(T, r, K, N)
    v = torch.zeros(T, r, device="cuda")
    a = c["x"], c["a"], c["b"], None
    y, good = torch.full_like(c["base"], 7), torch.empty_like(c["base"])
    order = c["order"].clone()
    gone = order[::3].long()
    order[::3] = torch.tensor([-1, T, 2**31 - 1], device="cuda", dtype=torch.int32).repeat(T)[
        :len(order[::3])]
    m.moe_adapters(*a, c["offsets"], order, c["base"], y, v, ws)
    m.moe_adapters(*a, c["offsets"], c["order"], c["base"], good, None, ws)
    torch.cuda.synchronize()
    stay = torch.ones(T, dtype=torch.bool, device="cuda")
    stay[gone] = False
    assert (y[gone] == 7).all() and torch.equal(y[stay], good[stay])
    dx, da, db = torch.full_like(c["x"], 7), torch.empty(3, r, K, device="cuda"), \
        torch.empty(3, r, N, device="cuda")
    m.moe_adapters_backward(c["dy"], c["x"], v, c["a"], c["b"], None, c["offsets"], order, dx, da,
                            db, ws)
    assert (dx[gone] == 7).all() and torch.isfinite(da).all() and torch.isfinite(db).all()
    for offsets in ([0, T, T + 5, 2**31 - 1], [-9, -5, 3, 2], [5, 5, 5, 5], [T, 0, T, 0]):
        off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
        m.moe_adapters(*a, off, c["order"], c["base"], y, v, ws)
        m.moe_adapters_backward(c["dy"], c["x"], v, c["a"], c["b"], None, off, c["order"], dx, da,
                                db, ws)
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("T", [90, 700])
@pytest.mark.parametrize("what", ["loud", float("nan"), float("inf")])
def test_an_adapter_changes_no_other_ones_results(m, T, dtype, what):
    r, K, N, J = 16, 1000, 1016, 5
    c = make(T, J, r, K, N, dtype)
    ws = m.adapters_workspace(T, r, K, N)

    def step():
        y, v = torch.empty_like(c["base"]), torch.zeros(T, r, device="cuda")
        dx, da, db = torch.empty_like(c["x"]), torch.empty(J, r, K, device="cuda"), \
            torch.empty(J, r, N, device="cuda")
        plan = c["scale"], c["offsets"], c["order"]
        m.moe_adapters(c["x"], c["a"], c["b"], *plan, c["base"], y, v, ws)
        m.moe_adapters_backward(c["dy"], c["x"], v, c["a"], c["b"], *plan, dx, da, db, ws)
        torch.cuda.synchronize()
        return y, dx, da, db

    good = step()
    one = c["ids"] == 2
    if what == "loud":
        c["scale"][2] = 2.0**40
        c["a"][2] *= 2**9
    else:
        c["x"][one], c["dy"][one] = what, what
    got = step()
    for p, q in zip(got[:2], good[:2]):
        assert torch.equal(p[~one], q[~one])
    rest = [0, 1, 3, 4]
    for p, q in zip(got[2:], good[2:]):
        assert torch.equal(p[rest], q[rest])


def same_infinities(got, want):
    """Elements that are not finite are the same infinities or NaN; want is in 64 bits."""
    got, want = got.double(), want.float().double()  # (what passes fp32's range is infinite)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(torch.isposinf(got), torch.isposinf(want))
    assert torch.equal(torch.isneginf(got), torch.isneginf(want))


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("T", [20, 1200])
def test_infinite_rows_give_infinities(m, T, dtype):
    """One rank, so that a sum has one infinity; by rows and in tiles alike."""
    K, N = 256, 136
    c = make(T, 3, 1, K, N, dtype, none=0.0)
    ws = m.adapters_workspace(T, 1, K, N)
    plan = c["scale"], c["offsets"], c["order"]
    f = {k: c[k].double() for k in ("x", "dy", "a", "b", "scale")}
    a, b, s = f["a"][c["ids"], 0], f["b"][c["ids"], 0], f["scale"][c["ids"], None]
    x, dy = c["x"].clone(), c["dy"].clone()
    x[5, 7], dy[9, 3] = float("inf"), float("-inf")
    y = torch.empty_like(c["base"])
    v = torch.zeros(T, 1, device="cuda")
    m.moe_adapters(x, c["a"], c["b"], *plan, c["base"], y, v, ws)
    want = c["base"].double() + s * (x.double() * a).sum(1, keepdim=True) * b
    assert torch.isinf(want[5]).sum() > N // 2 and torch.isfinite(want).sum() >= (T - 1) * N
    same_infinities(y, want)
    # gradients: u of one position is infinite
    m.moe_adapters(c["x"], c["a"], c["b"], *plan, c["base"], y, v, ws)
    dx, da, db = torch.empty_like(x), torch.empty(3, 1, K, device="cuda"), \
        torch.empty(3, 1, N, device="cuda")
    m.moe_adapters_backward(dy, c["x"], v, c["a"], c["b"], *plan, dx, da, db, ws)
    u = s * (dy.double() * b).sum(1, keepdim=True)
    assert torch.isinf(u).sum() == 1
    same_infinities(dx, u * a)
    for j in range(3):
        at = c["ids"] == j
        same_infinities(da[j, 0], (u[at] * f["x"][at]).sum(0))
    # (dy's own infinity meets v's terms: infinite or NaN, in its column only)
    j = int(c["ids"][9])
    assert not torch.isfinite(db[j, 0, 3])
    db[j, 0, 3] = 0
    assert torch.isfinite(db).all()


@pytest.mark.parametrize("r", [16, 100])
@pytest.mark.parametrize("T", [20, 1200])
def test_one_infinite_rank_among_finite_ones(m, T, r):
    K, N = 256, 136
    c = make(T, 3, r, K, N, BF16, none=0.0)
    j = int(c["ids"][5])
    c["x"][5, 7], c["a"][j, 0, 7] = 2.0**100, 2.0**40
    c["x"][6:, 7] = 0
    c["x"][:5, 7] = 0
    ws = m.adapters_workspace(T, r, K, N)
    y = torch.empty_like(c["base"])
    v = torch.zeros(T, r, device="cuda")
    m.moe_adapters(c["x"], c["a"], c["b"], c["scale"], c["offsets"], c["order"], c["base"], y, v, ws)
    assert torch.isinf(v).sum() == 1 and not torch.isnan(v).any()
    want = v[torch.argsort(c["order"])[5]].double() @ c["b"][j].double()
    assert torch.isinf(want).all()
    same_infinities(y[5], want)
    rest = torch.arange(T, device="cuda") != 5
    assert torch.isfinite(y[rest]).all()


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("r", [16, 64, 65, 128])
@pytest.mark.parametrize("T,K", [(400, 65536), (2500, 5120)])
def test_long_sums_are_rounded_on_the_way(m, T, K, r, dtype):
    """v of positive numbers, whose MMAs all cut off in one direction.

    Sixteen MMAs lose at most 2 u each of what is held then, 17 u of their sum for terms of
    about one size (16 + 15 + .. + 1 of 16, each 2 u); a CTA adds its chunks of 256 products
    rounded, u of the growing sum each; eight CTAs' parts and the store follow.  A sixteenth
    more covers chunks that are not alike.  One chain of MMAs would lose up to K / 16 u."""
    J, N = 2, 8
    c = make(T, J, r, K, N, dtype, none=0.0)
    c["x"], c["a"] = c["x"].abs() + 0.5, (c["a"].float().abs() + 0.5 / K**0.5).to(dtype)
    v = torch.zeros(T, r, device="cuda")
    y, ws = torch.empty_like(c["base"]), m.adapters_workspace(T, r, K, N)
    m.moe_adapters(c["x"], c["a"], c["b"], c["scale"], c["offsets"], c["order"], c["base"], y, v, ws)
    torch.cuda.synchronize()
    units = 17 + K / 256 / 2 / 8 + 8 + 1  # of u; the split over eight CTAs
    if T == 2500:
        units = 17 + K / 256 / 2 + 8 + 1  # not split, at most
    for j in range(J):
        at = torch.nonzero(c["ids"][c["order"].long()] == j)[:, 0]
        want = c["x"][c["order"][at].long()].double() @ c["a"][j].double().T
        off = ((v[at].double() - want).abs() / want).max()
        assert float(off) <= 17 / 16 * units * U, float(off) / U


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("which", ["all", "one"])
@pytest.mark.parametrize("T,J,r,K,N", [
    (500, 4096, 17, 40, 24), (460, 300, 64, 264, 520), (1000, 512, 128, 136, 72),
    (1300, 700, 16, 256, 264), (700, 400, 16, 256, 264), (450, 1000, 33, 72, 80)])
def test_many_loaded_adapters(m, T, J, r, K, N, which, dtype):
    """By rows while they are few beside the SMs, in tiles above, whatever number is loaded."""
    ids = None if which == "all" else torch.full((T,), J // 3, device="cuda")
    c = make(T, J, r, K, N, dtype, ids=ids)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    y, ws = torch.empty_like(c["base"]), m.adapters_workspace(T, r, K, N)
    before = m.launch_counts()["adapters"]
    m.moe_adapters(c["x"], c["a"], c["b"], c["scale"], c["offsets"], c["order"], c["base"], y, None, ws)
    by_rows = T <= (8 if r <= 16 else 3) * sms
    assert m.launch_counts()["adapters"] - before == (1 if by_rows else 2)
    check(m, c)


def row_form(T, J, r, K, N):
    """(CTAs, warps) of a position where the call goes by rows (adapters.cu: row_cluster, row_warps)."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    cluster = 1
    while cluster < 8 and max(K, N) >= 2 * cluster * 256:
        cluster *= 2
    warps = 4 if r <= 16 else 8 if r <= 32 else 16
    while warps > 4 and T * cluster * warps * 2 > 16 * sms:
        warps //= 2
    return cluster, warps


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("extra", [0, 8, 3])
@pytest.mark.parametrize("T,J,r,K,N,form", [
    (1, 2, 64, 5120, 1024, (8, 16)), (1, 1, 128, 2048, 2056, (8, 16)), (3, 8, 100, 1001, 515, (2, 16)),
    (8, 8, 33, 264, 520, (2, 16)), (2, 3, 65, 7, 3000, (8, 16)), (1, 1, 127, 200, 90, (1, 16)),
    (4, 4, 24, 1000, 1544, (4, 8)), (40, 30, 64, 1032, 600, (4, 4)), (30, 20, 48, 520, 1000, (2, 16)),
    (60, 50, 40, 600, 72, (2, 8)), (2, 2, 17, 4096, 4104, (8, 8)), (3, 2, 16, 4096, 264, (8, 4))])
def test_widths_of_a_row(m, T, J, r, K, N, form, extra, dtype):
    """Four, eight and sixteen warps a CTA, one to eight CTAs a row."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    if sms == 152:
        assert row_form(T, J, r, K, N) == form
    c = make(T, J, r, K, N, dtype, none=0.0 if T == 1 else 0.2)
    y, ws = torch.empty_like(c["base"]), m.adapters_workspace(T, r, K, N)
    before = m.launch_counts()["adapters"]
    m.moe_adapters(c["x"], c["a"], c["b"], c["scale"], c["offsets"], c["order"], c["base"], y, None, ws)
    assert m.launch_counts()["adapters"] - before == 1
    check(m, c, extra)


@pytest.mark.parametrize("r", [16, 64, 128])
def test_beside_the_layer(m, r):
    """Calls in turn with the layer's on one stream, whose kernels start before the last ones have
    ended, and beside them on another one: both hold tensor memory."""
    c = tiled(r, 1024, 1024, T=1500)
    spec = dict(hidden=1024, inter=512, n_routed=8, top_k=2, renormalize=True)
    cfg = m.config_from_spec(spec)
    T, g = c["T"], gen(7)
    w = [(randn(g, 8, *s) / 32).to(BF16) for s in ((512, 1024), (512, 1024), (1024, 512))]
    w_r = randn(g, 8, 1024) / 32
    lws = [m.workspace(cfg, T) for _ in range(2)]
    ws = [m.adapters_workspace(T, r, 1024, 1024) for _ in range(2)]
    out = [torch.empty_like(c["x"]) for _ in range(2)]
    y = [torch.empty_like(c["base"]) for _ in range(2)]

    def step(i, stream=None):
        m.moe_layer_forward(cfg, T, c["x"], w_r, None, *w, None, None, None, None, None, None,
                            out[i], lws[i], stream=stream)
        m.moe_adapters(out[i], c["a"], c["b"], c["scale"], c["offsets"], c["order"], c["base"], y[i],
                       None, ws[i], stream=stream)

    step(0)
    torch.cuda.synchronize()
    first = out[0].clone(), y[0].clone()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for i, s in enumerate(streams):
            step(i, s)
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(out[i], first[0]) and torch.equal(y[i], first[1])
