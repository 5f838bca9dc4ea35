"""An MoE block with 4-bit experts for decode, and a training step around sorted
tokens, built from the operators around the expert layer.

    python examples/w4_block.py

Decode: the residual addition and RMS norm give the router's rows in bf16 and
the experts' int8 codes with a scale per token; the picks are sorted by expert
and the codes travel with their scales; gate and up run as one 4-bit product
with SwiGLU, down as another; the weighted rows return to their tokens.  Every
buffer is allocated once and the step is replayed as a CUDA graph.

Training: the same routing, sorted tokens through bf16 experts in torch, and
gradients through the sort, the experts, the weights and the router.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import sparse_expert_layer_gb300 as moe  # noqa: E402
from sparse_expert_layer_gb300 import autograd  # noqa: E402


class W4Block:
    """x, residual -> (block output, new residual) for a fixed number of tokens."""

    def __init__(self, T, hidden, inter, n_experts, top_k, group=128, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.E, self.k = n_experts, top_k
        self.cfg = moe.config_from_spec(dict(hidden=hidden, inter=inter, n_routed=n_experts,
                                             top_k=top_k, renormalize=True))

        def matrix(n, k):  # random codes; scales as for weights of deviation 1 / sqrt(k)
            codes = torch.randint(0, 16, (n_experts, n, k), generator=g, device="cuda",
                                  dtype=torch.uint8)
            scales = (0.5 + torch.rand(n_experts, n, k // group, generator=g, device="cuda")) \
                / (4.6 * k**0.5)
            return moe.pack_w4(codes), scales.to(torch.bfloat16)

        self.gate, self.up = matrix(inter, hidden), matrix(inter, hidden)
        self.down = matrix(hidden, inter)
        self.gamma = torch.ones(hidden, dtype=torch.bfloat16, device="cuda")
        self.w_router = torch.randn(n_experts, hidden, generator=g, device="cuda") / hidden**0.5

        R = T * top_k
        bf16 = dict(dtype=torch.bfloat16, device="cuda")
        i32 = dict(dtype=torch.int32, device="cuda")
        f32 = dict(dtype=torch.float32, device="cuda")
        self.y = torch.empty(T, hidden, **bf16)
        self.q = torch.empty(T, hidden, dtype=torch.int8, device="cuda")
        self.q_scale = torch.empty(T, 1, **f32)
        self.ids, self.weights = torch.empty(T, top_k, **i32), torch.empty(T, top_k, **f32)
        self.counts, self.offsets = torch.empty(n_experts, **i32), torch.empty(n_experts + 1, **i32)
        self.s2e, self.e2s = torch.empty(R, **i32), torch.empty(R, **i32)
        self.q_sorted = torch.empty(R, hidden, dtype=torch.int8, device="cuda")
        self.scale_sorted = torch.empty(R, **f32)
        self.h = torch.empty(R, inter, **bf16)
        self.expert_out = torch.empty(R, hidden, **f32)
        self.out = torch.empty(T, hidden, **bf16)
        self.ws = moe.workspace(self.cfg, T)
        self.sort_ws = moe.sort_workspace(T, top_k, n_experts)

    def __call__(self, x, residual):
        """Updates residual in place and returns the block's output buffer."""
        moe.moe_add_rmsnorm(x, residual, self.gamma, 1e-6, residual, self.y, self.q, self.q_scale)
        moe.moe_route(self.cfg, x.shape[0], self.y, self.w_router, None, self.ids, self.weights,
                      self.ws)
        moe.moe_sort_tokens(self.E, self.ids, self.q, self.q_scale, self.counts, self.offsets,
                            self.s2e, self.e2s, self.q_sorted, self.scale_sorted, self.sort_ws)
        moe.moe_w4_gemv(self.q_sorted, self.scale_sorted, self.offsets, *self.gate, None, self.h,
                        *self.up)
        moe.moe_w4_gemv(self.h, None, self.offsets, *self.down, None, self.expert_out)
        moe.moe_unsort_tokens(self.expert_out, self.offsets, self.e2s, self.weights, self.out)
        return self.out


def expert_mlp(x_sorted, offsets, w_in, w_out):
    """A bf16 expert per slice of the sorted rows, in torch."""
    bounds = offsets.tolist()
    rows = [torch.nn.functional.silu(x_sorted[a:b] @ w_in[e]) @ w_out[e]
            for e, (a, b) in enumerate(zip(bounds[:-1], bounds[1:])) if b > a]
    return torch.cat(rows) if rows else x_sorted.new_zeros(0, w_out.shape[2])


def training_step(x, target, w_router, w_in, w_out, top_k):
    """Loss of one step; the gradients land in the leaves' .grad."""
    scores = torch.softmax(x.float() @ w_router.T, dim=-1)
    top = torch.topk(scores, top_k, dim=-1)
    weights = top.values / top.values.sum(-1, keepdim=True)
    x_sorted, plan = autograd.sort_tokens(x, top.indices.int(), w_router.shape[0])
    y_sorted = expert_mlp(x_sorted, plan.offsets, w_in, w_out)
    out = autograd.unsort_tokens(y_sorted, weights, plan, dtype=torch.float32)
    loss = torch.nn.functional.mse_loss(out, target)
    loss.backward()
    return loss.detach()


def decode(T=32, hidden=1024, inter=512, n_experts=32, top_k=4, steps=20):
    """Microseconds of a replayed step, the block, and its inputs' copies."""
    block = W4Block(T, hidden, inter, n_experts, top_k)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(T, hidden, generator=g, device="cuda").bfloat16()
    residual = torch.randn(T, hidden, generator=g, device="cuda").bfloat16()
    start = residual.clone()
    block(x, residual)  # outside the graph once: kernel attributes are set on first use
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block(x, residual)
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(steps):
        graph.replay()
    b.record()
    residual.copy_(start)
    graph.replay()
    torch.cuda.synchronize()
    if moe.moe_check_device_status(block.ws) != moe.MOE_OK:
        raise RuntimeError("the router reported a device error")
    return a.elapsed_time(b) * 1e3 / steps, block, x, start, residual


def train(T=256, hidden=256, inter=128, n_experts=8, top_k=2, steps=15):
    """Losses of a few steps of gradient descent, each a fixed share of a leaf's norm."""
    g = torch.Generator(device="cuda").manual_seed(2)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, target = rand(T, hidden).bfloat16(), rand(T, hidden)
    leaves = [(rand(n_experts, hidden) / hidden**0.5).requires_grad_(),
              (rand(n_experts, hidden, inter) / hidden**0.5).bfloat16().requires_grad_(),
              (rand(n_experts, inter, hidden) / inter**0.5).bfloat16().requires_grad_()]
    losses = []
    for _ in range(steps):
        losses.append(float(training_step(x, target, *leaves, top_k)))
        with torch.no_grad():
            for p in leaves:
                p -= 0.05 * p.norm() * p.grad / p.grad.norm()
                p.grad = None
    return losses


if __name__ == "__main__":
    us, *_ = decode()
    print(f"decode: {us:.1f} us a step")
    losses = train()
    print("training: loss " + " ".join(f"{v:.4f}" for v in losses[::7]))
