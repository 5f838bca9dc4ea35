"""A block for a few tokens of several requests, each with its own low-rank adapter, and the
fine-tuning of such adapters with clipped gradients.

    python examples/adapter_block.py

Decode: the residual addition and RMS norm, a projection in 4 bits that all requests share with
each request's adapter beside it, the second norm, and the expert layer for a few tokens with
4-bit experts.  Every buffer is allocated once and the step is replayed as a CUDA graph.

Training: adapters beside a frozen projection; one sort of the rows by adapter serves forward and
backward, the gradients are clipped by their global norm before they are applied.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import sparse_expert_layer_gb300 as moe  # noqa: E402
from sparse_expert_layer_gb300 import autograd  # noqa: E402


def _w4(g, *shape, group):
    """Random codes and scales as for weights of deviation 1 / sqrt(K)."""
    K = shape[-1]
    codes = torch.randint(0, 16, shape, generator=g, device="cuda", dtype=torch.uint8)
    scales = (0.5 + torch.rand(*shape[:-1], K // group, generator=g, device="cuda")) / (4.6 * K**0.5)
    return moe.pack_w4(codes), scales.to(torch.bfloat16)


class AdapterBlock:
    """x, residual, adapter ids -> (block output, new residual) for up to T tokens."""

    def __init__(self, T, hidden, inter, n_experts, top_k, n_adapters, rank=16, group=64, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        bf16 = dict(dtype=torch.bfloat16, device="cuda")
        i32 = dict(dtype=torch.int32, device="cuda")
        self.cfg = moe.config_from_spec(dict(hidden=hidden, inter=inter, n_routed=n_experts,
                                             top_k=top_k, renormalize=True, shared_inter=inter))
        self.weights = {}
        for m, n, k in (("gate", inter, hidden), ("up", inter, hidden), ("down", hidden, inter)):
            self.weights["w_" + m], self.weights["s_" + m] = _w4(g, n_experts, n, k, group=group)
            self.weights["shared_" + m], self.weights["s_shared_" + m] = _w4(g, n, k, group=group)
        self.w_router = torch.randn(n_experts, hidden, generator=g, device="cuda") / hidden**0.5
        self.experts = moe.FewTokenExperts(self.cfg, self.weights, self.w_router)
        self.proj = _w4(g, 1, hidden, hidden, group=group)
        self.a = (torch.randn(n_adapters, rank, hidden, generator=g, device="cuda")
                  / hidden**0.5).bfloat16()
        self.b = (0.5 * torch.randn(n_adapters, rank, hidden, generator=g, device="cuda")
                  / rank**0.5).bfloat16()
        self.scale = torch.full((n_adapters,), 2.0, device="cuda")
        self.gamma = torch.ones(hidden, **bf16)
        self.n_adapters = n_adapters

        self.y, self.p, self.y2, self.out = (torch.empty(T, hidden, **bf16) for _ in range(4))
        self.counts = torch.empty(n_adapters, **i32)
        self.offsets = torch.empty(n_adapters + 1, **i32)
        self.order, self.inverse = torch.empty(T, **i32), torch.empty(T, **i32)
        self.ids = torch.empty(T, top_k, **i32)
        self.picked = torch.empty(T, top_k, device="cuda")
        self.few_ws = moe.few_tokens_workspace(self.experts, T)
        self.adapter_ws = moe.adapters_workspace(T, rank, hidden, hidden)
        self.sort_ws = moe.sort_workspace(T, 1, n_adapters)

    def __call__(self, x, residual, adapter_ids):
        """adapter_ids int32 [T, 1]; updates residual in place, returns the output buffer."""
        moe.moe_sort_tokens(self.n_adapters, adapter_ids, None, None, self.counts, self.offsets,
                            self.order, self.inverse, None, ws=self.sort_ws)
        moe.moe_add_rmsnorm(x, residual, self.gamma, 1e-6, residual, self.y)
        moe.moe_w4_gemv(self.y, None, None, *self.proj, None, self.p)
        moe.moe_adapters(self.y, self.a, self.b, self.scale, self.offsets, self.order, self.p,
                         self.p, None, self.adapter_ws)
        moe.moe_add_rmsnorm(self.p, residual, self.gamma, 1e-6, residual, self.y2)
        moe.moe_few_tokens(self.experts, self.y2, self.out, self.few_ws, self.ids, self.picked)
        return self.out


def decode(T=4, hidden=1024, inter=512, n_experts=32, top_k=4, n_adapters=8, steps=20):
    """Microseconds of a replayed step, the block, and its inputs' copies."""
    block = AdapterBlock(T, hidden, inter, n_experts, top_k, n_adapters)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(T, hidden, generator=g, device="cuda").bfloat16()
    residual = torch.randn(T, hidden, generator=g, device="cuda").bfloat16()
    # the last token's request has no adapter
    ids = torch.randint(0, n_adapters, (T, 1), generator=g, device="cuda", dtype=torch.int32)
    ids[-1] = -1
    start = residual.clone()
    block(x, residual, ids)  # outside the graph once: kernel attributes are set on first use
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block(x, residual, ids)
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(steps):
        graph.replay()
    b.record()
    residual.copy_(start)
    graph.replay()
    torch.cuda.synchronize()
    if moe.moe_check_device_status(block.few_ws) != moe.MOE_OK:
        raise RuntimeError("the expert layer reported a device error")
    return a.elapsed_time(b) * 1e3 / steps, block, x, start, residual, ids


def tune(T=512, hidden=256, n_adapters=4, rank=8, steps=12, max_norm=0.5):
    """(losses, gradient norms before and after clipping) of a few steps that fit adapters to a
    projection they lack; rows of the last adapter id have none."""
    g = torch.Generator(device="cuda").manual_seed(3)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = rand(T, hidden).bfloat16()
    w = (rand(hidden, hidden) / hidden**0.5).bfloat16()
    ids = torch.randint(0, n_adapters + 1, (T,), generator=g, device="cuda", dtype=torch.int32)
    plan = autograd.plan_adapters(ids, n_adapters)
    missing = rand(n_adapters + 1, hidden, hidden) / hidden**0.5
    target = (x @ w.T).float() + 0.3 * torch.einsum("tk,tkn->tn", x.float(), missing[ids.long()])
    leaves = [(rand(n_adapters, rank, hidden) / hidden**0.5).bfloat16().requires_grad_(),
              torch.zeros(n_adapters, rank, hidden, device="cuda").bfloat16().requires_grad_()]
    ws, norm = moe.clip_workspace(), torch.empty(1, device="cuda")
    losses, norms = [], []
    for _ in range(steps):
        y = autograd.adapters(x @ w.T, x, *leaves, None, plan)
        loss = ((y.float() - target) ** 2).sum(-1).mean()
        loss.backward()
        grads = [p.grad for p in leaves]
        moe.moe_clip_grad_norm(grads, max_norm, norm, ws)
        after = sum(float((t.double() ** 2).sum()) for t in grads) ** 0.5
        norms.append((float(norm), after))
        losses.append(float(loss.detach()))
        with torch.no_grad():
            for p in leaves:
                p -= 0.1 * p.grad
                p.grad = None
    return losses, norms


if __name__ == "__main__":
    us, *_ = decode()
    print(f"decode: {us:.1f} us a step")
    losses, norms = tune()
    print("tuning: loss " + " ".join(f"{v:.4f}" for v in losses[::4]))
    print("gradient norms " + " ".join(f"{a:.3f}->{b:.3f}" for a, b in norms[::4]))
