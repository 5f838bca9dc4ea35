"""Measured cases of further operators: a whole layer for a few tokens, adapters, clipping.

Three operators: the expert layer from the router to the combined output for at
most eight tokens, with 16-bit or 4-bit experts (kind "few"); low-rank adapters
of many requests at once beside a shared projection (kind "adapt") and their
gradients ("adapt_grads"); the global norm of many gradients and their clipping
(kind "clip").

`run` with `own` false computes them in elementary torch operations, with
`own` true through the package's entry points.  `exact` computes the same
outputs in 64 bits from the definitions.
"""
from __future__ import annotations

import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = 1e-6


# ------------------------------------------------------------------- cases --
def _few(name, T, H, I, E, k, zero, shared, score, dtype, group, zeros):
    """group None: 16-bit weights, else 4-bit ones whose scales stand for that many channels."""
    return {"name": name, "kind": "few", "T": T, "H": H, "I": I, "E": E, "k": k, "zero": zero,
            "shared": shared, "score": score, "dtype": dtype, "bits": 16 if group is None else 4,
            "group": group or 0, "zeros": zeros}


def _adapt(name, kind, T, J, r, K, N, dtype, none):
    """none: share of the tokens without an adapter."""
    return {"name": name, "kind": kind, "T": T, "J": J, "r": r, "K": K, "N": N, "dtype": dtype,
            "none": none}


def _clip(name, count, least, most, dtype, clipped):
    return {"name": name, "kind": "clip", "count": count, "least": least, "most": most,
            "dtype": dtype, "clipped": clipped}


def listed():
    return [
        # one decoded token through a layer of 256 4-bit experts and a shared one: latency
        _few("few_one_token", 1, 7168, 2048, 256, 8, 0, 2048, "sigmoid", "bf16", 128, False),
        # a draft of eight tokens through 64 experts in bf16 and a wide shared expert
        _few("few_eight_tokens", 8, 5120, 1536, 64, 8, 0, 4096, "softmax", "bf16", None, False),
        # five tokens, small groups with zero points, a third of the picks pass through
        _few("few_zero_experts", 5, 2304, 736, 96, 6, 48, 0, "softmax", "fp16", 32, True),
        # one decoded token of one request with its own adapter: latency
        _adapt("adapt_one_token", "adapt", 1, 8, 16, 5120, 5120, "bf16", 0.0),
        # a decode batch of requests with 48 adapters, an eighth of them without one
        _adapt("adapt_decode", "adapt", 64, 48, 16, 7168, 2048, "bf16", 0.125),
        # a prefill chunk of a few requests
        _adapt("adapt_prefill", "adapt", 8192, 6, 64, 5120, 5120, "bf16", 0.0),
        # gradients of a small fp16 model with ragged sizes
        _adapt("adapt_grads_ragged", "adapt_grads", 333, 5, 24, 1000, 1544, "fp16", 0.2),
        # gradients of a training micro-batch over four adapters
        _adapt("adapt_grads_train", "adapt_grads", 8192, 4, 16, 7168, 5120, "bf16", 0.0),
        # the fp32 gradients of 24 adapters of rank 16: latency
        _clip("clip_adapters", 48, 16 * 2048, 16 * 7168, "fp32", True),
        # tensors from a bias to a matrix, of all types, whose norm is below the limit
        _clip("clip_mixed", 37, 5, 5120 * 1024, "mixed", False),
        # the gradients of 64 experts
        _clip("clip_experts", 3, 64 * 1536 * 5120, 64 * 1536 * 5120, "bf16", True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["few", "few", "few", "adapt", "adapt", "adapt_grads", "clip"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if kind == "few":
        T = rng.choice([1, 1, 2, 3, 4, 6, 8])
        H = 64 * _log(rng, 4, 112)
        I = 32 * _log(rng, 2, 64)
        group = rng.choice([None, None, 32, 64, 128, 0])
        if group and (H % group or I % group):
            group = 32
        size = 2.0 if group is None else 0.5
        E = rng.choice([8, 16, 64, 96, 128, 256])
        while E > 8 and E * I * H * size > 64 * 1536 * 5120 * 2:
            E //= 2
        k = min(rng.choice([1, 2, 4, 6, 8]), E // 2)
        while T > 1 and T * k * I * H > 64 * 1536 * 5120:
            T -= 1
        shared = rng.choice([0, 0, I, 2 * I])
        return {"kind": kind, "T": T, "H": H, "I": I, "E": E, "k": k,
                "zero": rng.choice([0, 0, E // 2]), "shared": shared,
                "score": rng.choice(["softmax", "sigmoid"]), "dtype": dtype,
                "bits": 16 if group is None else 4, "group": group or 0,
                "zeros": group is not None and rng.random() < 0.4}
    if kind == "clip":
        most = _log(rng, 1000, 20_000_000)
        return {"kind": kind, "count": min(_log(rng, 1, 60), 1 + 400_000_000 // most),
                "least": _log(rng, 1, most), "most": most,
                "dtype": rng.choice(["bf16", "fp16", "fp32", "mixed"]),
                "clipped": rng.random() < 0.7}
    r = rng.choice([4, 8, 16, 16, 24, 32, 64])
    K, N = _log(rng, 256, 7168), _log(rng, 256, 7168)
    if rng.random() < 0.8:
        K, N = max(8, K // 8 * 8), max(8, N // 8 * 8)
    T = _log(rng, 1, 8192)
    J = min(_log(rng, 1, 64), 512 // r)
    while T * r * (K + N) > 8192 * 16 * 12288 * 2:
        T //= 2
    return {"kind": kind, "T": T, "J": J, "r": r, "K": K, "N": N, "dtype": dtype,
            "none": rng.choice([0.0, 0.0, 0.25])}


# ------------------------------------------------------------------ inputs --
def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def _matrix(s, g, name, shape, bits, groups, dtype, zeros):
    """One stack of weights of deviation 1 / sqrt(K) under `name` (scales s_, zero points z_)."""
    K = shape[-1]
    if bits == 16:
        s["w"]["w_" + name] = (_randn(g, *shape) / K**0.5).to(dtype)
        return
    s["w"]["w_" + name] = torch.randint(0, 256, (*shape[:-1], K // 2), generator=g, device="cuda",
                                        dtype=torch.uint8)
    s["w"]["s_" + name] = ((0.5 + torch.rand(*shape[:-1], groups, generator=g, device="cuda"))
                           / (4.6 * K**0.5)).to(dtype)
    if zeros:
        s["w"]["z_" + name] = torch.randint(6, 10, (*shape[:-1], groups), generator=g,
                                            device="cuda", dtype=torch.uint8)


def _prepare_few(s, g):
    c = s["case"]
    T, H, I, E, k, dt = c["T"], c["H"], c["I"], c["E"], c["k"], DT[c["dtype"]]
    s["w_router"] = _randn(g, E + c["zero"], H) / H**0.5
    # of four candidates for each token, the one whose k-th pick is clearest
    x = _randn(g, 4 * T, H, dtype=dt)
    top = torch.sort(x.double() @ s["w_router"].double().T, dim=-1, descending=True).values
    best = (top[:, k - 1] - top[:, k]).view(4, T).argmax(0)
    s["x"] = x.view(4, T, H)[best, torch.arange(T, device="cuda")].contiguous()
    s["w"] = {}
    for name, n, m in (("gate", I, H), ("up", I, H), ("down", H, I)):
        groups = m // c["group"] if c["group"] else 1
        _matrix(s, g, name, (E, n, m), c["bits"], groups, dt, c["zeros"])
    if c["shared"]:
        for name, n, m in (("gate", c["shared"], H), ("up", c["shared"], H), ("down", H, c["shared"])):
            groups = m // c["group"] if c["group"] else 1
            _matrix(s, g, "shared_" + name, (n, m), c["bits"], groups, dt, c["zeros"])
    s["out"] = torch.empty(T, H, dtype=dt, device="cuda")
    return s


def _prepare_adapt(s, g):
    c = s["case"]
    T, J, r, K, N, dt = c["T"], c["J"], c["r"], c["K"], c["N"], DT[c["dtype"]]
    ids = torch.randint(0, J, (T,), generator=g, device="cuda")
    ids = torch.where(torch.rand(T, generator=g, device="cuda") < c["none"], J, ids)
    s["ids"] = ids
    s["order"] = torch.sort(ids, stable=True).indices.to(torch.int32)
    s["offsets"] = (ids[None, :] < torch.arange(J + 1, device="cuda")[:, None]).sum(1).to(
        torch.int32)
    s["x"] = _randn(g, T, K, dtype=dt)
    s["a"] = (_randn(g, J, r, K) / K**0.5).to(dt)
    s["b"] = (0.3 * _randn(g, J, r, N) / r**0.5).to(dt)
    s["scale"] = 0.5 + 1.5 * torch.rand(J, generator=g, device="cuda")
    if c["kind"] == "adapt":
        s["base"] = _randn(g, T, N, dtype=dt)
        s["y"] = torch.empty(T, N, dtype=dt, device="cuda")
        return s
    s["dy"] = (0.01 * _randn(g, T, N)).to(dt)
    # the forward pass has kept x A^T of the rows, in sorted order
    every = (s["x"].float() @ s["a"].float().view(J * r, K).T).view(T, J, r)
    picked = every[torch.arange(T, device="cuda"), ids.clamp(max=J - 1)] * (ids < J)[:, None]
    s["v"] = picked[s["order"].long()].contiguous()
    s["dx"] = torch.empty(T, K, dtype=dt, device="cuda")
    s["da"] = torch.empty(J, r, K, device="cuda")
    s["db"] = torch.empty(J, r, N, device="cuda")
    return s


def _sizes(c):
    """Sizes from the least to the most, evenly on their logarithm."""
    steps = max(1, c["count"] - 1)
    return [int(c["least"] * (c["most"] / c["least"]) ** (i / steps)) for i in range(c["count"])]


def _dtypes(c):
    if c["dtype"] == "mixed":
        return [("bf16", "fp32", "fp16")[i % 3] for i in range(c["count"])]
    return [c["dtype"]] * c["count"]


def _prepare_clip(s, g):
    c = s["case"]
    n = _sizes(c)
    s["grads"] = [_randn(g, m).mul_(0.01).to(DT[d]) for m, d in zip(n, _dtypes(c))]
    s["outs"] = [torch.empty_like(t) for t in s["grads"]]
    s["norm"] = torch.empty(1, device="cuda")
    # about a third of the norm, or about three times the norm
    s["max_norm"] = 0.01 * math.sqrt(sum(n)) * (0.35 if c["clipped"] else 3.0)
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    if case["kind"] == "few":
        return _prepare_few(s, g)
    return _prepare_clip(s, g) if case["kind"] == "clip" else _prepare_adapt(s, g)


# ------------------------------------------------------------- plain forms --
def _plain_route(s):
    """Picks [T, k] and their weights; logits in 64 bits, since a pick hangs on their order."""
    c = s["case"]
    logits = s["x"].double() @ s["w_router"].double().T
    if c["score"] == "softmax":
        e = torch.exp(logits - logits.amax(-1, keepdim=True))
        score = e / e.sum(-1, keepdim=True)
    else:
        score = 1.0 / (1.0 + torch.exp(-logits))
    top = torch.sort(score, dim=-1, descending=True, stable=True)
    w = top.values[:, :c["k"]]
    return top.indices[:, :c["k"]], (w / w.sum(-1, keepdim=True)).float()


def _plain_rows(w, name, pick):
    """The picked experts' matrices in 32 bits (pick None: the shared expert's)."""
    m = w["w_" + name] if pick is None else w["w_" + name][pick]
    if m.dtype != torch.uint8:
        return m.float()
    scale, zero = w["s_" + name], w.get("z_" + name)
    scale = (scale if pick is None else scale[pick]).float()[..., None]
    z = 8.0 if zero is None else (zero if pick is None else zero[pick]).float()[..., None]
    q = torch.stack([m & 15, m >> 4], dim=-1).view(*scale.shape[:-1], -1).float()
    return ((q - z) * scale).view(*m.shape[:-1], 2 * m.shape[-1])


def _silu(v):
    return v / (1.0 + torch.exp(-v))


def _plain_few(s):
    c = s["case"]
    T, k, E = c["T"], c["k"], c["E"]
    ids, weight = _plain_route(s)
    x = s["x"].float()
    pick = ids.reshape(-1).clamp(max=E - 1)
    rows = x.repeat_interleave(k, 0)[:, :, None]
    h = _silu(torch.bmm(_plain_rows(s["w"], "gate", pick), rows))
    h = h * torch.bmm(_plain_rows(s["w"], "up", pick), rows)
    y = torch.bmm(_plain_rows(s["w"], "down", pick), h)[:, :, 0].view(T, k, -1)
    y = torch.where((ids < E)[:, :, None], y, x[:, None, :])  # the others pass the token through
    out = (weight[:, :, None] * y).sum(1)
    if c["shared"]:
        h = _silu(x @ _plain_rows(s["w"], "shared_gate", None).T)
        h = h * (x @ _plain_rows(s["w"], "shared_up", None).T)
        out = out + h @ _plain_rows(s["w"], "shared_down", None).T
    return [out.to(DT[c["dtype"]])]


def _plain_own_columns(s, t):
    """t [T, J * r] with the columns of other adapters than a token's own zeroed."""
    J = s["case"]["J"]
    mine = s["ids"][:, None] == torch.arange(J, device="cuda")
    return torch.where(mine[:, :, None], t.view(len(t), J, -1), 0.0).view(len(t), -1)


def _plain_adapt(s):
    c = s["case"]
    J, r = c["J"], c["r"]
    v = _plain_own_columns(s, s["x"].float() @ s["a"].float().view(J * r, -1).T)
    v = v * s["scale"].repeat_interleave(r)
    y = s["base"].float() + v @ s["b"].float().view(J * r, -1)
    return [y.to(DT[c["dtype"]])]


def _plain_adapt_grads(s):
    c = s["case"]
    J, r, T = c["J"], c["r"], c["T"]
    scale = s["scale"].repeat_interleave(r)
    dy, x, a = s["dy"].float(), s["x"].float(), s["a"].float().view(J * r, -1)
    u = _plain_own_columns(s, dy @ s["b"].float().view(J * r, -1).T) * scale
    v = torch.empty_like(s["v"])
    v[s["order"].long()] = s["v"]
    v = _plain_own_columns(s, v[:, None, :].expand(T, J, r).reshape(T, J * r)) * scale
    dx = u @ a
    return [dx.to(DT[c["dtype"]]), (u.T @ x).view(J, r, -1), (v.T @ dy).view(J, r, -1)]


def _plain_clip(s):
    total = torch.stack([(t.float() ** 2).sum(dtype=torch.float64) for t in s["grads"]]).sum()
    norm = torch.sqrt(total)
    c = torch.clamp(s["max_norm"] / (norm + EPS), max=1.0).float()
    return [norm.float().view(1)] + [(t.float() * c).to(t.dtype) for t in s["grads"]]


# -------------------------------------------------------- the package's calls --
def _own_few(s, moe):
    c = s["case"]
    if "experts" not in s:  # the handle and the workspace that a program keeps
        cfg = moe.config_from_spec(dict(
            hidden=c["H"], inter=c["I"], n_routed=c["E"], n_zero=c["zero"], top_k=c["k"],
            score=c["score"], renormalize=True, shared_inter=c["shared"]))
        named = {n.replace("w_shared_", "shared_"): t for n, t in s["w"].items()}
        s["experts"] = moe.FewTokenExperts(cfg, named, s["w_router"])
        s["ws"] = moe.few_tokens_workspace(s["experts"], c["T"])
    moe.moe_few_tokens(s["experts"], s["x"], s["out"], s["ws"])
    return [s["out"]]


def _own_adapt(s, moe):
    c = s["case"]
    if "ws" not in s:
        s["ws"] = moe.adapters_workspace(c["T"], c["r"], c["K"], c["N"])
    moe.moe_adapters(s["x"], s["a"], s["b"], s["scale"], s["offsets"], s["order"], s["base"],
                     s["y"], None, s["ws"])
    return [s["y"]]


def _own_adapt_grads(s, moe):
    c = s["case"]
    if "ws" not in s:
        s["ws"] = moe.adapters_workspace(c["T"], c["r"], c["K"], c["N"])
    moe.moe_adapters_backward(s["dy"], s["x"], s["v"], s["a"], s["b"], s["scale"], s["offsets"],
                              s["order"], s["dx"], s["da"], s["db"], s["ws"])
    return [s["dx"], s["da"], s["db"]]


def _own_clip(s, moe):
    if "ws" not in s:
        s["list"] = moe.TensorList(s["grads"], s["outs"])
        s["ws"] = moe.clip_workspace()
    moe.moe_clip_grad_norm(s["list"], s["max_norm"], s["norm"], s["ws"], EPS)
    return [s["norm"]] + s["outs"]


def run(state):
    kind = state["case"]["kind"]
    if own:
        import sparse_expert_layer_gb300 as moe

        return {"few": _own_few, "adapt": _own_adapt, "adapt_grads": _own_adapt_grads,
                "clip": _own_clip}[kind](state, moe)
    return {"few": _plain_few, "adapt": _plain_adapt, "adapt_grads": _plain_adapt_grads,
            "clip": _plain_clip}[kind](state)


# -------------------------------------------------------------------- work --
def work(case):
    c = case
    if c["kind"] == "few":
        T, H, I, b = c["T"], c["H"], c["I"], SIZE[c["dtype"]]
        all_ids = c["E"] + c["zero"]
        picks = T * c["k"] * c["E"] / all_ids  # of experts with weights, on average
        hit = c["E"] * (1 - (1 - c["k"] / all_ids) ** T)  # distinct ones, on average
        def matrix(n, m):
            if c["bits"] == 16:
                return n * m * b
            groups = m // c["group"] if c["group"] else 1
            return n * m // 2 + n * groups * (b + (1 if c["zeros"] else 0))
        data = 4 * all_ids * H + 2 * T * H * b + int(hit * (2 * matrix(I, H) + matrix(H, I)))
        if c["shared"]:
            data += 2 * matrix(c["shared"], H) + matrix(H, c["shared"])
        return {"bytes": data, "flops": int(2 * T * all_ids * H + 6 * picks * H * I
                                            + 6 * T * H * c["shared"])}
    if c["kind"] == "clip":
        n = _sizes(c)
        return {"bytes": sum(2 * m * SIZE[d] for m, d in zip(n, _dtypes(c))), "flops": 3 * sum(n)}
    T, r, K, N, b = c["T"], c["r"], c["K"], c["N"], SIZE[c["dtype"]]
    rows = T * (1 - c["none"])
    hit = c["J"] * (1 - (1 - (1 - c["none"]) / c["J"]) ** T)  # adapters with tokens, on average
    ab = hit * r * (K + N) * b
    if c["kind"] == "adapt":
        return {"bytes": int(rows * K * b + 2 * T * N * b + ab + 8 * T),
                "flops": int(2 * rows * r * (K + N))}
    return {"bytes": int(rows * (K + N) * b + T * K * b + 4 * rows * r + ab
                         + 4 * c["J"] * r * (K + N) + 8 * T),
            "flops": int(4 * rows * r * (K + N))}


# ------------------------------------------------------------- in 64 bits --
def _exact_matrix(w, name, e):
    m = w["w_" + name] if e is None else w["w_" + name][e]
    if m.dtype != torch.uint8:
        return m.double()
    scale, zero = w["s_" + name], w.get("z_" + name)
    scale = (scale if e is None else scale[e]).double()
    packed = m.to(torch.int64)
    q = torch.empty(m.shape[0], 2 * m.shape[1], dtype=torch.float64, device="cuda")
    q[:, 0::2] = (packed % 16).double()
    q[:, 1::2] = (packed // 16).double()
    width = q.shape[1] // scale.shape[1]
    q -= 8 if zero is None else (zero if e is None else zero[e]).double().repeat_interleave(width, 1)
    return q * scale.repeat_interleave(width, 1)


def _exact_swiglu(w, prefix, e, x):
    g = _exact_matrix(w, prefix + "gate", e) @ x
    h = g * torch.sigmoid(g) * (_exact_matrix(w, prefix + "up", e) @ x)
    return _exact_matrix(w, prefix + "down", e) @ h


def _exact_few(s):
    c = s["case"]
    wr = s["w_router"].double()
    out = torch.zeros(c["T"], c["H"], dtype=torch.float64, device="cuda")
    for t in range(c["T"]):
        x = s["x"][t].double()
        logit = wr @ x
        score = torch.softmax(logit, 0) if c["score"] == "softmax" else torch.sigmoid(logit)
        best = torch.topk(score, c["k"])
        share = (best.values / best.values.sum()).tolist()
        for e, p in zip(best.indices.tolist(), share):
            out[t] += p * (_exact_swiglu(s["w"], "", e, x) if e < c["E"] else x)
        if c["shared"]:
            out[t] += _exact_swiglu(s["w"], "shared_", None, x)
    return [out]


def _segments(s):
    bounds, order = s["offsets"].tolist(), s["order"].long()
    return [(j, bounds[j], bounds[j + 1], order[bounds[j]:bounds[j + 1]])
            for j in range(s["case"]["J"]) if bounds[j] < bounds[j + 1]]


def _exact_adapt(s):
    y = s["base"].double()
    for j, _, _, rows in _segments(s):
        y[rows] += float(s["scale"][j]) * (s["x"][rows].double() @ s["a"][j].double().T
                                           @ s["b"][j].double())
    return [y]


def _exact_adapt_grads(s):
    dx = torch.zeros(s["dx"].shape, dtype=torch.float64, device="cuda")
    da = torch.zeros(s["da"].shape, dtype=torch.float64, device="cuda")
    db = torch.zeros(s["db"].shape, dtype=torch.float64, device="cuda")
    for j, lo, hi, rows in _segments(s):
        scaled = float(s["scale"][j]) * s["dy"][rows].double()
        u = scaled @ s["b"][j].double().T
        dx[rows] = u @ s["a"][j].double()
        da[j] = torch.einsum("tr,tk->rk", u, s["x"][rows].double())
        db[j] = torch.einsum("tr,tn->rn", s["v"][lo:hi].double(), scaled)
    return [dx, da, db]


def _exact_clip(s):
    total = sum(float(torch.dot(t.double(), t.double())) for t in s["grads"])
    norm = math.sqrt(total)
    c = min(1.0, s["max_norm"] / (norm + EPS))
    return [torch.tensor([norm], dtype=torch.float64)] + [t.double() * c for t in s["grads"]]


def exact(case, seed):
    s = prepare(case, seed)
    return {"few": _exact_few, "adapt": _exact_adapt, "adapt_grads": _exact_adapt_grads,
            "clip": _exact_clip}[case["kind"]](s)
