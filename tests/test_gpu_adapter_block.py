"""The operators together, as examples/adapter_block.py uses them: a decode step of requests with
their own adapters as one graph, each step checked on its inputs in 64 bits, and a few steps of
fine-tuning with clipped gradients."""
import importlib.util
import os

import pytest
import torch

from tests import gpu_support as gs
from tests import test_gpu_few_tokens as few

pytestmark = pytest.mark.gpu

U = 2.0**-24
BF16 = torch.bfloat16
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    gs.lib()
    path = os.path.join(ROOT, "examples", "adapter_block.py")
    spec = importlib.util.spec_from_file_location("adapter_block", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def within(got, want, tol, what):
    over = (got.double() - want).abs() - tol
    assert float(over.max()) <= 0, f"{what}: {float(over.max()):.3e} more than allowed"


def half_step(t):
    return 2.0**-8 * t.abs() + 2.0**-134


@pytest.mark.parametrize("T", [1, 4, 8])
def test_decode_block(ex, T):
    us, block, x, start, residual, ids = ex.decode(T=T)
    assert us > 0
    H = x.shape[1]
    r = x.double() + start.double()

    def norm(v):
        return v / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-6)

    within(block.y, norm(r), half_step(norm(r)) + 32 * U * norm(r).abs(), "first norm")
    # the projection and each token's adapter on the norm's output
    packed, scales = block.proj[0][0], block.proj[1][0]
    q = torch.stack([packed & 15, packed >> 4], -1).view(H, H).double() - 8
    w = q * scales.double().repeat_interleave(64, 1)
    y = block.y.double()
    base, size = y @ w.T, y.abs() @ w.abs().T
    tol = (H / 8 + 64) * U * size + half_step(base)  # rounded to bf16 before the adapter
    want = base.clone()
    for t, j in enumerate(ids[:, 0].tolist()):
        if j >= 0:
            d = 2.0 * (block.a[j].double() @ y[t]) @ block.b[j].double()
            want[t] += d
            tol[t] += 2.0**-12 * (2.0 * (block.a[j].double().abs() @ y[t].abs())
                                  @ block.b[j].double().abs())
    within(block.p, want, tol + half_step(want), "projection with adapters")
    # the second norm takes the first sum as it was rounded
    r1 = r.to(BF16).double()
    r2 = block.p.double() + r1
    within(residual, r2, half_step(r2) + U * r2.abs(), "residual")
    within(block.y2, norm(r2), half_step(norm(r2)) + 32 * U * norm(r2).abs(), "second norm")
    # the expert layer on its own picks, which the router's tests check
    spec = dict(n_routed=32, hidden=H, shared_inter=512)
    out, tol = few.exact(dict(spec=spec, x=block.y2, w=block.weights, bits=4, dtype=BF16),
                         block.ids.cpu(), block.picked.double().cpu())
    within(block.out, out, tol, "expert layer")


def test_tuning(ex):
    losses, norms = ex.tune()
    assert all(v == v for v in losses) and len(losses) == 12
    assert any(before > 0.5 for before, _ in norms)
    for before, after in norms:
        want = min(before, 0.5)
        # each element is rounded to bf16 once more
        assert abs(after - want) <= 2.0**-8 * want + 1e-6
