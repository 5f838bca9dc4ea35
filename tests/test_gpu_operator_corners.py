"""Corners of the operators around the layer: values at the ends of the fp32
range, tensors that autograd watches, plans and ids of any layout."""
import pytest
import torch

from tests import gpu_support as gs

pytestmark = pytest.mark.gpu

U = 2.0**-24
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
INT8, E4M3 = torch.int8, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def m():
    return gs.lib()


def gen(seed=0):
    return torch.Generator(device="cuda").manual_seed(seed)


def strided(t, extra):
    """The same matrix with `extra` further channels between its rows."""
    wide = torch.full((t.shape[0], t.shape[1] + extra), 5.0, device=t.device, dtype=t.dtype)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


def norm_codes(m, x, qdt, group, eps=1e-6, gamma=None):
    """(y, codes as fp32, scale) of a norm without a residual."""
    T, H = x.shape
    y = torch.full((T, H), 7.0, device="cuda", dtype=x.dtype)
    q = torch.full((T, H), 7, device="cuda", dtype=INT8).view(qdt)
    scale = torch.full((T, -(-H // group) if group else 1), -1.0, device="cuda")
    m.moe_add_rmsnorm(x, None, gamma, eps, None, y, q, scale, group)
    torch.cuda.synchronize()
    return y, q.to(FP32), scale


# ------------------------------------------------- norm: rows of tiny values --
# Whole numbers p of at most 127 times 2^e, 127 in every group and zeros between:
# the codes are known without rounding.  int8: p itself.  e4m3: p * 448 / 127,
# which lies at least 2^-10 of itself away from the middle of two codes unless it
# is one of them, so an fp32 error does not change it.
TINY = [(FP32, -149), (FP32, -133), (BF16, -133), (FP32, -103), (FP32, -102), (FP32, -60),
        (BF16, -60)]


@pytest.mark.parametrize("dtype,e", TINY)
@pytest.mark.parametrize("H,extra", [(256, 0), (256, 8), (256, 3), (255, 0), (257, 0), (33, 0),
                                     (2056, 0), (2051, 0)])
@pytest.mark.parametrize("qdt", [INT8, E4M3])
@pytest.mark.parametrize("group", [0, 32, 256])
def test_codes_of_tiny_rows(m, dtype, e, H, extra, qdt, group):
    g = gen(H + group)
    p = torch.randint(-127, 128, (3, H), generator=g, device="cuda").double()
    p[torch.rand(3, H, generator=g, device="cuda") < 0.2] = 0
    p[:, ::32] = 127
    p[1, ::32] = -127
    p[2] = 0
    p[2, H - 1] = 127  # one channel alone; its row has groups of zeros
    x = (p * 2.0**e).to(dtype)
    assert torch.equal(x.double(), p * 2.0**e)
    if extra:
        x = strided(x, extra)
    _, code, scale = norm_codes(m, x, qdt, group)
    want = p if qdt == INT8 else (p * 448 / 127).to(FP32).to(E4M3).double()
    assert torch.equal(code.double(), want)
    # scale = max|y| / most: the mean and its root within 32 u (halved), two
    # products and the rounded 1 / most, each a step of the subnormals at worst
    width = group or H
    G = scale.shape[1]
    rms = torch.sqrt((x.double() ** 2).mean(-1, keepdim=True) + 1e-6)
    amax = torch.nn.functional.pad(x.double().abs(), (0, G * width - H)).view(3, G, width).amax(-1)
    want = amax / rms / (127 if qdt == INT8 else 448)
    assert ((scale.double() - want).abs() <= 36 * U * want + 2.0**-149).all()


# ------------------------------------- norm: the ends of the fp32 statistics --
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("H", [64, 256, 257, 1000, 7161])
@pytest.mark.parametrize("qdt", [INT8, E4M3])
@pytest.mark.parametrize("group", [0, 32])
def test_zero_rows_without_eps(m, dtype, H, qdt, group):
    x = torch.randn(4, H, generator=gen(H), device="cuda").to(dtype)
    rest = [norm_codes(m, x, qdt, group, eps=0.0)]
    x[1] = 0
    x[3] = -0.0
    y, code, scale = norm_codes(m, x, qdt, group, eps=0.0)
    for t in (y, code, scale):
        assert (t[[1, 3]] == 0).all()
    for got, before in zip((y, code, scale), rest[0]):
        assert torch.equal(got[[0, 2]], before[[0, 2]]) and torch.isfinite(got).all()


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("H", [256, 257, 4100])
@pytest.mark.parametrize("group", [0, 32])
def test_rows_past_the_range_of_the_squares_show(m, dtype, H, group):
    x = torch.ones(5, H, device="cuda", dtype=dtype)
    x[1] = 2.0**66
    x[2, 7] = -(2.0**64)
    x[4] = 2.0**56  # squares of 2^112: inside
    y, _, scale = norm_codes(m, x, INT8, group)
    assert torch.isnan(y[[1, 2]]).all() and torch.isnan(scale[[1, 2]]).all()
    for r in (0, 3, 4):
        assert ((y[r].double() - 1).abs() <= 2.0**-8 + 32 * U).all()
        assert ((scale[r].double() * 127 - 1).abs() <= 2.0**-19).all()


@pytest.mark.parametrize("H", [256, 257])
def test_rows_whose_squares_vanish_show_without_eps(m, H):
    # 2^-90 squared is below fp32: nothing is left to divide by
    x = torch.full((2, H), 2.0**-90, device="cuda")
    x[:, 3] = 0
    y, code, scale = norm_codes(m, x, INT8, 0, eps=0.0)
    assert torch.isinf(scale).all() and not torch.isfinite(y).any()
    y, code, scale = norm_codes(m, x, INT8, 0, eps=1e-20)
    want = x.double() * 1e10
    assert ((y.double() - want).abs() <= 32 * U * want).all()
    assert torch.equal(code, 127 * (x > 0).float())


def test_norm_of_as_many_rows_as_an_int_counts(m):
    # the last rows' successors lie past 2^31 - 1
    T = 2**31 - 1
    x = torch.zeros(T, 1, device="cuda", dtype=BF16)
    x[-30000:] = torch.randn(30000, 1, generator=gen(), device="cuda").to(BF16)
    out = torch.full((T, 1), 7.0, device="cuda", dtype=BF16)
    m.moe_add_rmsnorm(x, None, None, 1e-6, out)
    torch.cuda.synchronize()
    assert torch.equal(out, x)


# ------------------------------------ 4 bits: rows of scales of every alignment --
@pytest.mark.parametrize("K,group", [(256, 32), (768, 32), (2304, 32), (128, 32), (1152, 64),
                                     (768, 64), (1088, 64), (512, 64), (256, 128), (768, 128),
                                     (1920, 128), (96, 0)])
@pytest.mark.parametrize("xdt,sdt", [(FP16, FP16), (BF16, FP32), (INT8, FP32), (INT8, BF16)])
def test_w4_groups_of_every_alignment(m, K, group, xdt, sdt):
    from tests.test_gpu_operators import check_w4, w4_case

    g = gen(K + group)
    check_w4(m, w4_case(g, 3, 13, 137, K, group, xdt, sdt, False, True), FP32)
    check_w4(m, w4_case(g, 2, 5, 70, K, group, xdt, sdt, True, True), BF16)


# ------------------------------------------------ tensors that autograd watches --
def raw_calls(m, g, T=20, k=2, E=4, H=64):
    """name -> (call, the tensors that it writes)."""
    i32 = dict(dtype=torch.int32, device="cuda")
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, res, y, out, dx = (rand(T, H) for _ in range(5))
    q, qs = torch.zeros(T, H, device="cuda", dtype=INT8), rand(T, 1)
    ids = torch.randint(0, E, (T, k), generator=g, **i32)
    plan = [torch.zeros(n, **i32) for n in (E, E + 1, T * k, T * k)]
    rows, dy, xsc = rand(T * k, H), rand(T * k, H), rand(T)
    ss, w, dw = rand(T * k), rand(T, k), rand(T, k)
    wq = torch.zeros(E, 8, H // 2, device="cuda", dtype=torch.uint8)
    wide, xw, one = rand(T * k, 8), rand(T * k, H).to(BF16), torch.ones(E, 8, 1, device="cuda")
    m.moe_sort_tokens(E, ids, None, None, *plan, None)
    return {
        "norm": (lambda: m.moe_add_rmsnorm(x, res, None, 1e-6, res, y, q, qs), (res, y, q, qs)),
        "sort": (lambda: m.moe_sort_tokens(E, ids, x, xsc, *plan, rows, ss), (*plan, rows, ss)),
        "sort_backward": (lambda: m.moe_sort_tokens_backward(rows, plan[1], plan[3], k, dx), (dx,)),
        "unsort": (lambda: m.moe_unsort_tokens(rows, plan[1], plan[3], w, out), (out,)),
        "unsort_backward": (lambda: m.moe_unsort_tokens_backward(out, rows, plan[1], plan[3], w, dy,
                                                                 dw), (dy, dw)),
        "w4": (lambda: m.moe_w4_gemv(xw, None, plan[1], wq, one, None, wide), (wide,)),
    }


CALLS = ["norm", "sort", "sort_backward", "unsort", "unsort_backward", "w4"]


@pytest.mark.parametrize("name", CALLS)
def test_written_tensors_count_as_changed(m, name):
    call, written = raw_calls(m, gen(1))[name]
    before = [t._version for t in written]
    call()
    torch.cuda.synchronize()
    assert all(t._version > v for t, v in zip(written, before))


@pytest.mark.parametrize("name", CALLS)
def test_written_tensors_may_not_require_a_gradient(m, name):
    call, written = raw_calls(m, gen(2))[name]
    for t in (t for t in written if t.is_floating_point() and t.dtype == FP32):
        before = t.clone()
        t.requires_grad_()
        with pytest.raises(ValueError, match="requires a gradient"):
            call()
        torch.cuda.synchronize()
        assert torch.equal(t.detach(), before)
        with torch.no_grad():  # as torch's own in-place calls
            call()
        t.requires_grad_(False)
    torch.cuda.synchronize()


def test_a_saved_residual_written_in_place_is_noticed(m):
    g = gen(3)
    x, res = (torch.randn(4, 64, generator=g, device="cuda") for _ in range(2))
    w = torch.ones(64, device="cuda", requires_grad=True)
    loss = (res * w).sum()  # keeps res for w's gradient
    m.moe_add_rmsnorm(x, res, None, 1e-6, res)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_inference_tensors_may_be_written(m):
    with torch.inference_mode():
        x = torch.ones(4, 64, device="cuda")
        m.moe_add_rmsnorm(x, None, None, 1e-6, None, x)
    m.moe_add_rmsnorm(x, None, None, 1e-6, None, x)
    torch.cuda.synchronize()
    assert (x.double() - 1).abs().max() <= 1e-6


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("T", [40, 700])
def test_frozen_expert_outputs_get_no_gradient(m, dtype, T):
    from sparse_expert_layer_gb300 import autograd

    k, E, H = 4, 8, 1024
    g = gen(T)
    ids = torch.randint(-1, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    _, plan = autograd.sort_tokens(torch.zeros(T, H, device="cuda", dtype=dtype), ids, E)
    y = torch.randn(T * k, H, generator=g, device="cuda").to(dtype)
    w = torch.rand(T, k, generator=g, device="cuda")
    grad = torch.randn(T, H, generator=g, device="cuda").to(dtype)
    grads, peaks = [], []
    for frozen in (False, True):
        yi, wi = y.clone().requires_grad_(not frozen), w.clone().requires_grad_()
        out = autograd.unsort_tokens(yi, wi, plan)
        torch.cuda.synchronize()
        start = torch.cuda.memory_allocated()
        torch.cuda.reset_peak_memory_stats()
        out.backward(grad)
        torch.cuda.synchronize()
        peaks.append(torch.cuda.max_memory_allocated() - start)
        grads.append(wi.grad)
        assert (yi.grad is None) == frozen
    assert torch.equal(*grads)
    rows = T * k * H * y.element_size()
    assert peaks[1] < rows <= peaks[0]


def test_the_gradient_of_the_rows_may_be_left_out(m):
    from tests.test_gpu_operators import back_case

    t, _, _, _ = back_case(gen(5), 50, 4, 8, 333, FP32, BF16, 4)
    args = t["dout"], t["y"], t["offsets"], t["e2s"], t["w"]
    dy, dw, alone = torch.empty_like(t["y"]), torch.empty_like(t["w"]), torch.empty_like(t["w"])
    m.moe_unsort_tokens_backward(*args, dy, dw)
    m.moe_unsort_tokens_backward(*args, None, alone)
    torch.cuda.synchronize()
    assert torch.equal(dw, alone)


@pytest.mark.parametrize("layout", ["columns", "transposed", "start", "expanded"])
def test_ids_of_any_layout_are_sorted(m, layout):
    from sparse_expert_layer_gb300 import autograd

    T, k, E, H = 30, 2, 8, 64
    g = gen(4)
    x = torch.randn(T, H, generator=g, device="cuda")
    draw = lambda *s: torch.randint(-1, E, s, generator=g, device="cuda",  # noqa: E731
                                    dtype=torch.int32)
    ids = {"columns": lambda: draw(T, k + 3)[:, 1:1 + k], "transposed": lambda: draw(k, T).T,
           "start": lambda: draw(T * k + 1)[1:].view(T, k),
           "expanded": lambda: draw(T, 1).expand(T, k)}[layout]()
    want, plan = autograd.sort_tokens(x, ids.clone(memory_format=torch.contiguous_format), E)
    got, other = autograd.sort_tokens(x, ids, E)
    assert torch.equal(got, want)
    assert torch.equal(plan.expanded_to_sorted, other.expanded_to_sorted)
    assert torch.equal(plan.offsets, other.offsets)
