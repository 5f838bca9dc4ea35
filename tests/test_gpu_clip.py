"""moe_clip_grad_norm against its definition in 64 bits.

Norm: a thread adds at most 16 squares in each of four fp32 accumulators, which two
additions join (18 u of a sum of positive terms, u = 2^-24), the rest is added as pairs of
fp32 (2^-44) and rounded once; the root halves that and is rounded once: 10.5 u.  Products: c adds a sum, a quotient and
the product, 14 u, and the rounding to the type.
"""
import math

import pytest
import torch

from tests import gpu_support as gs

pytestmark = pytest.mark.gpu

U = 2.0**-24
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
TINY = {BF16: 2.0**-134, FP16: 2.0**-25, FP32: 2.0**-150}
EPS = 1e-6


@pytest.fixture(scope="module")
def m():
    return gs.lib()


def gen(seed=0):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, dtype=FP32):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def norm_of(tensors):
    return math.sqrt(sum(float((t.double() ** 2).sum()) for t in tensors))


def check(m, tensors, max_norm, outs=None, what=""):
    """Runs the call and compares norm and outputs with the definition."""
    kept = [t.clone() for t in tensors]
    norm = torch.full((1,), -1.0, device="cuda")
    lst = m.TensorList(tensors, outs)
    m.moe_clip_grad_norm(lst, max_norm, norm, m.clip_workspace(), EPS)
    torch.cuda.synchronize()
    want = norm_of(kept)
    assert abs(float(norm) - want) <= 11 * U * want, (what, float(norm), want)
    c = min(1.0, max_norm / (want + EPS))
    for t, k, o in zip(tensors, kept, lst.outs):
        if o is None or k.numel() == 0:
            continue
        if max_norm > (want + EPS) * (1 + 20 * U):
            assert torch.equal(o, k), what
        else:
            y = k.double() * c
            tol = (torch.finfo(o.dtype).eps / 2 + 14 * U) * y.abs() + TINY[o.dtype]
            assert ((o.double() - y).abs() <= tol).all(), what
        if o is not t:
            assert torch.equal(t, k), what


SIZES = [1, 2, 7, 8, 9, 31, 2047, 2048, 16383, 16384, 16385, 100003]


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("n", SIZES)
def test_one_tensor(m, dtype, n):
    t = randn(gen(n), n, dtype=dtype)
    norm = norm_of([t])
    check(m, [t.clone()], 0.3 * norm)
    check(m, [t.clone()], 0.3 * norm, [torch.full_like(t, 7)])
    check(m, [t.clone()], 3 * norm)
    check(m, [t.clone()], 3 * norm, [torch.full_like(t, 7)])


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("at,to", [(1, 1), (3, 5), (0, 1), (7, 0), (2, 2), (8, 4)])
@pytest.mark.parametrize("n", [1, 5, 8, 16385])
def test_views_that_start_anywhere(m, dtype, at, to, n):
    g = gen(at + n)
    flat = randn(g, at + n + 11, dtype=dtype)
    into = torch.full((to + n + 13,), 7.0, device="cuda", dtype=dtype)
    before = flat.clone()
    check(m, [flat[at:at + n]], 0.5 * norm_of([flat[at:at + n]]), [into[to:to + n]])
    assert torch.equal(flat, before)
    assert (into[:to] == 7).all() and (into[to + n:] == 7).all()
    check(m, [flat[at:at + n]], 0.5 * norm_of([flat[at:at + n]]))
    assert torch.equal(flat[:at], before[:at]) and torch.equal(flat[at + n:], before[at + n:])


@pytest.mark.parametrize("count", [2, 48, 49, 512, 513, 1300])
def test_many_tensors(m, count):
    g = gen(count)
    tensors = []
    for i in range(count):
        n = [0, 1, 130, 4099, 20000][i % 5] if i % 7 else 33
        tensors.append(randn(g, n, dtype=(BF16, FP16, FP32)[i % 3]) * (1 + i % 4))
    norm = norm_of(tensors)
    check(m, tensors, 0.1 * norm)
    check(m, tensors, 10 * norm)
    check(m, tensors, 0.05 * norm, [None if i % 2 else torch.empty_like(t)
                                    for i, t in enumerate(tensors)])


def test_shapes_lists_and_no_tensors(m):
    ws = m.clip_workspace()
    norm = torch.full((1,), -1.0, device="cuda")
    m.moe_clip_grad_norm([], 1.0, norm, ws)
    assert float(norm) == 0.0
    m.moe_clip_grad_norm([torch.zeros(0, device="cuda")], 1.0, norm, ws)
    assert float(norm) == 0.0
    t = [torch.full((2, 3, 4), 2.0, device="cuda"), torch.tensor(5.0, device="cuda")]
    m.moe_clip_grad_norm(t, 1.0, norm, ws)  # in place
    assert float(norm) == 11.0 and abs(float(t[1]) - 5 / 11) < 1e-6
    zero = torch.zeros(100, device="cuda")
    m.moe_clip_grad_norm([zero], 1.0, norm, ws)
    assert float(norm) == 0.0 and (zero == 0).all()
    m.moe_clip_grad_norm([t[0]], 0.0, None, ws)
    assert (t[0] == 0).all()
    m.moe_clip_grad_norm(m.TensorList([t[1]], [None]), 0.0, norm, ws)  # only the norm
    assert abs(float(norm) - 5 / 11) < 1e-6 and float(t[1]) != 0


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
def test_what_is_not_finite(m, dtype):
    ws = m.clip_workspace()
    norm = torch.empty(1, device="cuda")
    a, b = torch.ones(1000, device="cuda", dtype=dtype), torch.ones(9, device="cuda")
    a[3] = float("inf")
    m.moe_clip_grad_norm([a, b], 1.0, norm, ws)
    assert float(norm) == float("inf")
    assert torch.isnan(a[3]) and (a[4:] == 0).all() and (b == 0).all()
    a[3] = float("nan")
    b.fill_(1)
    m.moe_clip_grad_norm([a, b], 1.0, norm, ws)
    assert math.isnan(float(norm)) and torch.isnan(a).all() and torch.isnan(b).all()


def test_ends_of_the_range(m):
    big = torch.full((50,), 2.0**63, device="cuda")  # squares of 2^126
    big[1:] = 2.0**60
    check(m, [big], 1.0)
    small = torch.full((5000,), 2.0**-62, device="cuda")
    norm = torch.empty(1, device="cuda")
    m.moe_clip_grad_norm(m.TensorList([small], [None]), 1.0, norm, m.clip_workspace())
    assert abs(float(norm) / norm_of([small]) - 1) <= 11 * U


def test_the_same_bits_on_every_call_and_in_a_graph(m):
    g = gen(3)
    src = [randn(g, n, dtype=d) for n, d in ((3000001, BF16), (77777, FP32), (5, FP16))]
    outs = [torch.empty_like(t) for t in src]
    norm, ws = torch.empty(1, device="cuda"), m.clip_workspace()
    lst = m.TensorList(src, outs)
    m.moe_clip_grad_norm(lst, 5.0, norm, ws)
    first = [norm.clone()] + [o.clone() for o in outs]
    for _ in range(3):
        ws.fill_(255)  # need not be initialised
        m.moe_clip_grad_norm(lst, 5.0, norm, ws)
        assert all(torch.equal(a, b) for a, b in zip(first, [norm] + outs))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.moe_clip_grad_norm(lst, 5.0, norm, ws)
    for t in outs + [norm]:
        t.fill_(7)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, [norm] + outs))
    src[1].mul_(2)  # a replay reads what the gradients hold then
    graph.replay()
    torch.cuda.synchronize()
    assert abs(float(norm) - norm_of(src)) <= 11 * U * norm_of(src)


def test_two_streams_at_once(m):
    g = gen(4)
    sets = [[randn(g, 4000001)], [3 * randn(g, 5000011)]]
    want = [norm_of(s) for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    state = [(m.TensorList(s, [torch.empty_like(s[0])]), torch.empty(1, device="cuda"),
              m.clip_workspace()) for s in sets]
    torch.cuda.synchronize()
    for _ in range(5):
        for st, (lst, norm, ws) in zip(streams, state):
            m.moe_clip_grad_norm(lst, 1.0, norm, ws, stream=st)
    torch.cuda.synchronize()
    for (lst, norm, _), w in zip(state, want):
        assert abs(float(norm) - w) <= 11 * U * w
        assert abs(norm_of(lst.outs) - 1) < 1e-5


def test_more_elements_than_an_int_counts(m):
    n = 2**31 + 9
    t = torch.zeros(n, device="cuda", dtype=BF16)
    t[0], t[-1], t[2**31 - 1] = 3.0, 4.0, 12.0
    norm = torch.empty(1, device="cuda")
    m.moe_clip_grad_norm([t], 6.5, norm, m.clip_workspace(), 0.0)
    torch.cuda.synchronize()
    assert float(norm) == 13.0
    assert float(t[0]) == 1.5 and float(t[-1]) == 2.0 and float(t[2**31 - 1]) == 6.0


def test_autograd_sees_what_was_written(m):
    w = torch.ones(10, device="cuda", requires_grad=True)
    ws = m.clip_workspace()
    with pytest.raises(ValueError, match="requires a gradient"):
        m.moe_clip_grad_norm([w], 1.0, None, ws)
    with torch.no_grad():
        m.moe_clip_grad_norm([w], 1.0, None, ws)
    x = torch.ones(10, device="cuda")
    y = (w * x).sum()
    m.moe_clip_grad_norm([x], 1.0, None, ws)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


def test_launches(m):
    t = [torch.ones(10, device="cuda")]
    before = m.launch_counts()
    m.moe_clip_grad_norm(t, 1.0, None, m.clip_workspace())
    after = m.launch_counts()
    assert after["grad_norm"] - before["grad_norm"] == 1 and after["clip"] - before["clip"] == 1


def test_the_factor_is_rounded_once(m):
    """Ones whose sums are exact: the norm is the root of their number, an output the factor."""
    import numpy as np

    ws, norm = m.clip_workspace(), torch.empty(1, device="cuda")
    for max_norm, eps in ((0.75, EPS), (3.0, 0.0), (0.1, 2.0**-3)):
        for n in list(range(10, 200)) + [777, 4096, 100003, 999999]:
            t = torch.ones(n, device="cuda")
            m.moe_clip_grad_norm([t], max_norm, norm, ws, eps)
            root = math.sqrt(n)
            c = float(np.float32(max_norm)) / (root + float(np.float32(eps)))
            # half a step, and the pair's own error
            assert abs(float(norm) - root) <= 0.501 * np.spacing(np.float32(root)), n
            assert abs(float(t[-1]) - c) <= 0.501 * np.spacing(np.float32(c)), n
            assert (t == t[0]).all()


def test_ends_of_the_factor(m):
    ws, norm = m.clip_workspace(), torch.empty(1, device="cuda")
    top = torch.finfo(FP32).max
    for value, max_norm, eps, want in ((2.0**60, 1.0, 0.0, 1.0), (2.0**-60, 2.0**-61, 0.0, 2.0**-61),
                                       (1.0, top, 0.0, 1.0), (1.0, 0.0, EPS, 0.0),
                                       (1.0, 1.0, top, 0.0), (4.0, 2.0**-140, 0.0, 2.0**-140)):
        t = torch.zeros(100, device="cuda")
        t[17] = value
        m.moe_clip_grad_norm([t], max_norm, norm, ws, eps)
        assert abs(float(t[17]) - want) <= 2.0**-23 * want + 2.0**-127, (value, max_norm, eps)
        assert float(norm) == value and torch.count_nonzero(t) <= 1
    t = torch.zeros(100, device="cuda")
    m.moe_clip_grad_norm([t], 0.0, norm, ws, 0.0)
    assert float(norm) == 0 and torch.isnan(t).all()  # 0 / 0
    t = torch.zeros(100, device="cuda")
    m.moe_clip_grad_norm([t], 1.0, norm, ws, 0.0)
    assert float(norm) == 0 and (t == 0).all()
