"""Timing cases of the operators of a training step around the layer: layer norm, linear maps with a fused
epilogue, the balance loss with the router's gradient, the global gradient norm with clipping.

  lnorm    h = x + residual, y = (h - mean h) / std(h) w + b in one pass, and its backward pass
  linear   y = act(x W^T + bias) + residual, optionally with z = x W^T + bias kept for training; backward:
           dz = dy act'(z) and the bias's gradient
  balance  the balance loss of a routed batch per sequence with per-expert counts; backward: the gradient of
           the router's logits from the mixture weights' gradient and the loss's
  clip     the 2-norm over many gradient tensors, and the tensors scaled to at most a given norm

A case is a dict of plain values; prepare() makes its inputs on the GPU from a seed, run() makes one pass
through the operator (in elementary float32 operations, or through the library when `own` is set), exact()
evaluates the definition in float64 and work() counts what a pass cannot do without.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


def listed():
    return [
        # One token of a GLM-5-wide decoder: the residual added and the next block's norm. Latency.
        {"name": "lnorm_step", "op": "lnorm", "dir": "fwd", "N": 1, "D": 6144, "dtype": "bf16", "res": True},
        # A prompt of 8,191 tokens of the GLM-4.5 width.
        {"name": "lnorm_prefill", "op": "lnorm", "dir": "fwd", "N": 8191, "D": 5120, "dtype": "bf16", "res": True},
        # Training step of the Air width: gradients of the rows, the weight and the bias.
        {"name": "lnorm_backward", "op": "lnorm", "dir": "bwd", "N": 4096, "D": 4096, "dtype": "bf16", "res": True},
        # One token through the first map of a dense FFN of the GLM-4.5 dense width: a weight stream.
        {"name": "linear_token", "op": "linear", "dir": "fwd", "N": 1, "K": 5120, "M": 12288, "act": "gelu_tanh",
         "res": False, "keep": False, "dtype": "bf16"},
        # A ragged batch through the second map, with the residual stream added.
        {"name": "linear_batch", "op": "linear", "dir": "fwd", "N": 201, "K": 12288, "M": 5120, "act": "none",
         "res": True, "keep": False, "dtype": "bf16"},
        # Training forward of the first map on 8,191 tokens: the pre-activation is kept.
        {"name": "linear_train", "op": "linear", "dir": "fwd", "N": 8191, "K": 5120, "M": 12288, "act": "gelu",
         "res": False, "keep": True, "dtype": "bf16"},
        # A float32 evaluation of 1,000 tokens.
        {"name": "linear_f32", "op": "linear", "dir": "fwd", "N": 1000, "K": 1536, "M": 4096, "act": "silu",
         "res": True, "keep": False, "dtype": "f32"},
        # Gradients behind the activation of 4,096 tokens, and the bias's.
        {"name": "linear_backward", "op": "linear", "dir": "bwd", "N": 4096, "M": 12288, "act": "gelu", "dtype": "bf16"},
        # Loss and counts of 8,192 tokens in eight sequences over GLM-5's 256 experts, padded at their ends.
        {"name": "balance_loss", "op": "balance", "dir": "fwd", "N": 8192, "E": 256, "k": 8, "T": 1024, "pad": True},
        # Gradient of the logits of 8,000 tokens over the GLM-4.5 experts, one sequence.
        {"name": "balance_backward", "op": "balance", "dir": "bwd", "N": 8000, "E": 160, "k": 8, "T": 8000,
         "pad": False},
        # Gradients of a small model part: norm weights, biases, a router. Latency.
        {"name": "clip_small", "op": "clip", "tensors": 7, "total": 1597697, "dtype": "f32", "to": "f32",
         "flat": False, "clips": True},
        # Gradients of a layer of experts kept as bfloat16, the clipped ones in float32 for the optimizer.
        {"name": "clip_layer", "op": "clip", "tensors": 56, "total": 290000001, "dtype": "bf16", "to": "f32",
         "flat": True, "clips": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _wide(rng, lo, hi, step=64):
    """A multiple of step between lo and hi, spread over the logarithm."""
    return max(1, int(round(_log(rng, lo, hi) / step))) * step


def draw(rng):
    op = rng.choice(["lnorm", "lnorm", "linear", "linear", "linear", "balance", "balance", "clip"])
    if op == "lnorm":
        c = {"op": op, "dir": rng.choice(["fwd", "bwd"]), "N": _log(rng, 1, 8192), "D": _wide(rng, 64, 8192, 8),
             "dtype": rng.choice(["bf16", "bf16", "f32"]), "res": rng.random() < 0.5}
        while c["N"] * c["D"] > (1 << 24) * (2 if c["dtype"] == "bf16" and c["dir"] == "fwd" else 1):
            c["N"] = c["N"] * 2 // 3
        return c
    if op == "linear":
        if rng.random() < 0.25:
            c = {"op": op, "dir": "bwd", "N": _log(rng, 1, 8192), "M": _wide(rng, 64, 16384, 8),
                 "act": rng.choice(ACTS), "dtype": rng.choice(["bf16", "bf16", "f32"])}
            while c["N"] * c["M"] > (1 << 25) * (2 if c["dtype"] == "bf16" else 1):
                c["N"] = c["N"] * 2 // 3
            return c
        f32 = rng.random() < 0.2
        c = {"op": op, "dir": "fwd", "N": _log(rng, 1, 8192), "K": _wide(rng, 256, 2048 if f32 else 12288),
             "M": _wide(rng, 64, 4096 if f32 else 16384, 8), "act": rng.choice(ACTS), "res": rng.random() < 0.5,
             "keep": rng.random() < 0.3, "dtype": "f32" if f32 else "bf16"}
        while c["N"] * c["K"] * c["M"] > 500000000000 // (64 if f32 else 1):
            c["N"] = c["N"] * 2 // 3
        return c
    if op == "balance":
        E = rng.choice([8, 16, 60, 64, 128, 160, 256, 288, 512])
        N = _log(rng, 1, 32768)
        return {"op": op, "dir": rng.choice(["fwd", "bwd"]), "N": N, "E": E, "k": min(E, rng.choice([1, 2, 4, 6, 8])),
                "T": max(1, rng.choice([N, _log(rng, 1, N), _log(rng, max(1, N // 16), N)])), "pad": rng.random() < 0.5}
    return {"op": op, "tensors": _log(rng, 1, 300), "total": _log(rng, 1 << 12, 1 << 27),
            "dtype": rng.choice(["bf16", "f32"]), "to": rng.choice(["bf16", "f32"]), "flat": rng.random() < 0.5,
            "clips": rng.random() < 0.8}


def _sizes(c):
    """Elements of each tensor: the total dealt out unevenly, a few tensors of one to a few values among them."""
    n, total = c["tensors"], c["total"]
    share = [math.exp(-9.0 * ((i * 0.6180339887) % 1.0)) for i in range(n)]
    sizes = [max(1, int(total * v / sum(share))) for v in share]
    for i in range(6, n, 7):
        sizes[i] = 1 + i % 5
    sizes[0] += max(0, total - sum(sizes))
    return sizes


# ---- inputs ----
def _randn(g, shape, dtype, std=1.0, mean=0.0):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).mul_(std).add_(mean).to(dtype)


def _tensors(g, case, dtype, fill):
    """Tensors of the case's sizes: each its own, or views of one flat buffer that lie end to end in it."""
    sizes = _sizes(case)
    if not case["flat"]:
        return [_randn(g, n, dtype, 0.02) if fill else torch.empty(n, dtype=dtype, device=DEV) for n in sizes]
    flat = torch.empty(sum(sizes), dtype=dtype, device=DEV)
    parts = list(flat.split(sizes))
    if fill:
        for p in parts:
            p.copy_(_randn(g, p.shape, dtype, 0.02))
    return parts


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    st = {"case": dict(case), "ws": None}
    f = {"dtype": torch.float32, "device": DEV}
    op = case["op"]
    if own:
        import sparse_moe_layer_gate_amd as moe
    if op == "lnorm":
        N, D, dt = case["N"], case["D"], TYPES[case["dtype"]]
        st["w"] = _randn(g, D, dt, 0.1, 1.0)
        st["b"] = _randn(g, D, dt, 0.1)
        if case["dir"] == "fwd":
            st["x"] = _randn(g, (N, D), dt, 2.0, 0.3)
            st["res"] = _randn(g, (N, D), dt, 2.0) if case["res"] else None
            st["h"] = torch.empty((N, D), dtype=dt, device=DEV) if case["res"] else None
            st["y"] = torch.empty((N, D), dtype=dt, device=DEV)
            st["stats"] = torch.empty((N, 2), **f)
        else:
            st["h"] = _randn(g, (N, D), dt, 2.0, 0.3)
            st["dy"] = _randn(g, (N, D), dt)
            st["dres"] = _randn(g, (N, D), dt) if case["res"] else None
            h = st["h"].double()  # what the forward call left
            st["stats"] = torch.stack((h.mean(1), (h.var(1, unbiased=False) + EPS).rsqrt()), 1).float()
            st["out"] = (torch.empty_like(st["h"]), torch.empty(D, **f), torch.empty(D, **f))
            if own:
                n = moe.moe_layer_norm_workspace_size(N, D, case["dtype"])
                st["ws"] = torch.empty(max(n, 256), dtype=torch.uint8, device=DEV)
    elif op == "linear":
        N, M, dt = case["N"], case["M"], TYPES[case["dtype"]]
        if case["dir"] == "fwd":
            K = case["K"]
            st["x"] = _randn(g, (N, K), dt)
            st["w"] = _randn(g, (M, K), dt, 1.0 / math.sqrt(K))
            st["bias"] = _randn(g, M, dt, 0.1)
            st["res"] = _randn(g, (N, M), dt) if case["res"] else None
            st["z"] = torch.empty((N, M), dtype=dt, device=DEV) if case["keep"] else None
            st["y"] = torch.empty((N, M), dtype=dt, device=DEV)
            if own:
                n = moe.moe_linear_workspace_size(N, K, M, case["dtype"])
                st["ws"] = torch.empty(max(n, 256), dtype=torch.uint8, device=DEV)
        else:
            st["dy"] = _randn(g, (N, M), dt)
            st["z"] = _randn(g, (N, M), dt)
            st["out"] = (torch.empty_like(st["dy"]), torch.empty(M, **f))
            if own:
                n = moe.moe_linear_backward_workspace_size(N, M, case["dtype"])
                st["ws"] = torch.empty(max(n, 256), dtype=torch.uint8, device=DEV)
    elif op == "balance":
        N, E, k, T = case["N"], case["E"], case["k"], case["T"]
        S = (N + T - 1) // T
        logits = torch.randn((N, E), generator=g, **f) + 0.5 * torch.randn((1, E), generator=g, **f)
        st["scores"] = torch.sigmoid(logits)
        st["idx"] = logits.topk(k, dim=1).indices.to(torch.int32)
        st["mask"] = None
        if case["pad"]:  # each sequence padded behind its own length
            length = torch.randint(0, T + 1, (S,), generator=g, device=DEV)
            n = torch.arange(N, device=DEV)
            st["mask"] = (n % T < length[n // T]).to(torch.uint8)
        st["alpha"], st["weight"] = 2.5, 1e-4
        if case["dir"] == "fwd":
            st["counts"] = torch.empty((S, E), dtype=torch.int32, device=DEV)
            st["coef"] = torch.empty((S, E), **f)
            st["loss"] = torch.empty(1, **f)
        else:
            st["coef"] = torch.rand((S, E), generator=g, **f) / T
            st["dw"] = torch.randn((N, k), generator=g, **f)
            st["dloss"] = torch.full((1,), 0.5, **f)
            st["out"] = torch.empty((N, E), **f)
        if own:
            st["cfg"] = moe.make_config(64, E, 1, 1, k, 64, alpha=st["alpha"])
            n = moe.moe_balance_workspace_size(st["cfg"], N, T)
            st["ws"] = torch.empty(max(n, 256), dtype=torch.uint8, device=DEV)
    else:
        st["grads"] = _tensors(g, case, TYPES[case["dtype"]], True)
        st["out"] = _tensors(g, case, TYPES[case["to"]], False)
        st["max"] = 0.5 * 0.02 * math.sqrt(case["total"]) if case["clips"] else 1e6
        st["norm"] = torch.empty(1, **f)
        if own:
            st["list"], st["to"] = moe.moe_tensor_list(st["grads"]), moe.moe_tensor_list(st["out"])
            st["ws"] = torch.empty(moe.moe_grad_norm_workspace_size(st["list"]), dtype=torch.uint8, device=DEV)
    return st


# ---- one pass ----
def run(st):
    c = st["case"]
    return globals()[("_own_" if own else "_plain_") + c["op"]](st, c)


def _own_lnorm(st, c):
    import sparse_moe_layer_gate_amd as moe

    if c["dir"] == "fwd":
        moe.moe_layer_norm(c["N"], st["x"], st["res"], st["w"], st["b"], st["h"], st["y"], st["stats"], eps=EPS)
        return (st["y"], st["stats"]) if st["h"] is None else (st["h"], st["y"], st["stats"])
    dh, dw, db = st["out"]
    moe.moe_layer_norm_backward(c["N"], st["h"], st["stats"], st["w"], st["dres"], st["dy"], dh, dw, db, st["ws"])
    return dh, dw, db


def _own_linear(st, c):
    import sparse_moe_layer_gate_amd as moe

    if c["dir"] == "fwd":
        moe.moe_linear(st["x"], st["w"], st["y"], st["ws"], bias=st["bias"], residual=st["res"], act=c["act"],
                       z=st["z"])
        return st["y"] if st["z"] is None else (st["y"], st["z"])
    dz, db = st["out"]
    moe.moe_linear_backward(st["dy"], st["z"], dz, db, st["ws"], act=c["act"])
    return dz, db


def _own_balance(st, c):
    import sparse_moe_layer_gate_amd as moe

    if c["dir"] == "fwd":
        moe.moe_balance_loss(st["cfg"], c["N"], st["scores"], st["idx"], c["T"], st["weight"], st["counts"],
                             st["coef"], st["loss"], st["ws"], token_mask=st["mask"])
        return st["loss"], st["counts"], st["coef"]
    moe.moe_route_backward(st["cfg"], c["N"], st["scores"], st["idx"], st["dw"], st["out"], seq_rows=c["T"],
                           coef=st["coef"], dloss=st["dloss"], token_mask=st["mask"])
    return st["out"]


def _own_clip(st, c):
    import sparse_moe_layer_gate_amd as moe

    moe.moe_grad_norm(st["list"], st["norm"], st["ws"])
    moe.moe_grad_clip(st["list"], st["norm"], st["max"], out=st["to"])
    return [st["norm"]] + st["out"]


def _plain_lnorm(st, c):
    dt = TYPES[c["dtype"]]
    if c["dir"] == "fwd":
        h = st["x"].float()
        if st["res"] is not None:
            h = h + st["res"].float()
        mean = h.mean(1, keepdim=True)
        d = h - mean
        rstd = torch.rsqrt((d * d).mean(1, keepdim=True) + EPS)
        y = (d * rstd * st["w"].float() + st["b"].float()).to(dt)
        stats = torch.cat((mean, rstd), 1)
        return (y, stats) if st["res"] is None else (h.to(dt), y, stats)
    mean, rstd = st["stats"][:, :1], st["stats"][:, 1:]
    n = (st["h"].float() - mean) * rstd
    dy = st["dy"].float()
    t = dy * st["w"].float()
    dh = rstd * (t - t.mean(1, keepdim=True) - n * (t * n).mean(1, keepdim=True))
    if st["dres"] is not None:
        dh = dh + st["dres"].float()
    return dh.to(dt), (dy * n).sum(0), dy.sum(0)


def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).float()
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if act == "gelu_tanh":
        a = math.sqrt(2.0 / math.pi)
        t = torch.tanh(a * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * a * (1.0 + 3.0 * 0.044715 * z * z)
    return torch.ones_like(z)


def _plain_linear(st, c):
    dt = TYPES[c["dtype"]]
    if c["dir"] == "fwd":
        z = st["x"].float().mm(st["w"].float().t()) + st["bias"].float()
        y = _act(z, c["act"])
        if st["res"] is not None:
            y = y + st["res"].float()
        return y.to(dt) if st["z"] is None else (y.to(dt), z.to(dt))
    dz = st["dy"].float() * _act_slope(st["z"].float(), c["act"])
    return dz.to(dt), dz.sum(0)


def _plain_balance(st, c):
    N, E, k, T = c["N"], c["E"], c["k"], c["T"]
    S = (N + T - 1) // T
    s = st["scores"]
    seq = torch.arange(N, device=DEV) // T
    live = torch.ones(N, device=DEV) if st["mask"] is None else st["mask"].float()
    p = s / s.sum(1, keepdim=True)
    if c["dir"] == "fwd":
        tokens = torch.zeros(S, device=DEV).index_add_(0, seq, live)
        # whole numbers, each exact in float32 up to 2^24
        chosen = torch.zeros((N, E), device=DEV).scatter_(1, st["idx"].long(), 1.0) * live[:, None]
        pad = S * T - N
        rows = torch.cat((chosen, chosen.new_zeros((pad, E)))).view(S, T, E)
        counts = rows.sum(1)
        rows = torch.cat((p * live[:, None], p.new_zeros((pad, E)))).view(S, T, E)
        some = torch.clamp(tokens, min=1.0)[:, None]
        mean = rows.sum(1) / some
        f = counts * E / (k * some)
        loss = st["weight"] / S * (f * mean).sum()
        return loss.view(1), counts.to(torch.int32), st["weight"] / S * f / some
    i = st["idx"].long()
    chosen = s.gather(1, i)
    total = chosen.sum(1, keepdim=True) + 1e-20
    dw = st["dw"]
    back = st["alpha"] / total * (dw - (dw * chosen).sum(1, keepdim=True) / total)
    ds = torch.zeros_like(s).scatter_add_(1, i, back)
    coef = st["coef"][seq]
    pull = (coef - (coef * p).sum(1, keepdim=True)) / s.sum(1, keepdim=True)
    ds = ds + st["dloss"] * live[:, None] * pull
    return ds * s * (1.0 - s)


def _plain_clip(st, c):
    total = torch.stack([g.float().square().sum(dtype=torch.float64) for g in st["grads"]]).sum()
    norm = total.sqrt().float().view(1)
    scale = torch.clamp(st["max"] / (norm + 1e-6), max=1.0)
    return [norm] + [(g.float() * scale).to(TYPES[c["to"]]) for g in st["grads"]]


# ---- what a pass cannot do without ----
def work(c):
    op = c["op"]
    if op == "clip":
        n = sum(_sizes(c))
        a, b = (4 if c[t] == "f32" else 2 for t in ("dtype", "to"))
        return {"bytes": n * (a + b), "flops": 3 * n}
    if op == "balance":
        N, E, k = c["N"], c["E"], c["k"]
        S = (N + c["T"] - 1) // c["T"]
        mask = N if c["pad"] else 0
        if c["dir"] == "fwd":
            return {"bytes": 4 * N * (E + k) + mask + 8 * S * E, "flops": 3 * N * E}
        return {"bytes": 4 * N * (2 * E + 2 * k) + mask + 4 * S * E, "flops": 10 * N * E}
    es = 4 if c["dtype"] == "f32" else 2
    N = c["N"]
    if op == "lnorm":
        D = c["D"]
        if c["dir"] == "fwd":
            return {"bytes": es * (N * D * (4 if c["res"] else 2) + 2 * D) + 8 * N, "flops": 9 * N * D}
        return {"bytes": es * (N * D * (4 if c["res"] else 3) + D) + 8 * N + 8 * D, "flops": 15 * N * D}
    M = c["M"]
    if c["dir"] == "bwd":
        return {"bytes": es * 3 * N * M + 4 * M, "flops": 12 * N * M}
    K = c["K"]
    return {"bytes": es * (N * K + M * K + M + N * M * (1 + c["res"] + c["keep"])), "flops": 2 * N * K * M}


# ---- the definitions in float64 ----
def exact(case, seed):
    st = prepare(case, seed)
    return globals()["_exact_" + case["op"]](st, case)


def _exact_lnorm(st, c):
    """Row blocks of the definition; the gradients from autograd of it."""
    N, D = c["N"], c["D"]
    w, b = st["w"].double(), st["b"].double()
    if c["dir"] == "fwd":
        hs, ys, ss = [], [], []
        for i in range(0, N, 2048):
            h = st["x"][i:i + 2048].double()
            if st["res"] is not None:
                h = torch.add(h, st["res"][i:i + 2048].double())
            var, mean = torch.var_mean(h, dim=1, correction=0)
            std = torch.sqrt(var + EPS)
            hs.append(h)
            ys.append(torch.addcmul(b, (h - mean[:, None]) / std[:, None], w))
            ss.append(torch.stack((mean, 1.0 / std), 1))
        out = (torch.cat(hs), torch.cat(ys), torch.cat(ss))
        return out if st["res"] is not None else out[1:]
    w.requires_grad_()
    b.requires_grad_()
    dh = []
    for i in range(0, N, 2048):
        h = st["h"][i:i + 2048].double().requires_grad_()
        centred = h - h.sum(1, keepdim=True) / D
        y = centred / torch.sqrt(centred.square().sum(1, keepdim=True) / D + EPS) * w + b
        y.backward(st["dy"][i:i + 2048].double())
        dh.append(h.grad if st["dres"] is None else h.grad + st["dres"][i:i + 2048].double())
    return torch.cat(dh), w.grad, b.grad


def _curve(z, act):
    """The activation in float64, differentiable; the normal distribution's own function for its two tails."""
    if act == "relu":
        return torch.clamp(z, min=0.0)
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return z * torch.special.ndtr(z)
    if act == "gelu_tanh":  # (1 + tanh u) / 2 = sigmoid(2 u)
        return z * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z.pow(3)))
    return z * 1.0


def _exact_linear(st, c):
    N, M = c["N"], c["M"]
    if c["dir"] == "fwd":
        wt = st["w"].double()
        ys, zs = [], []
        for i in range(0, N, 2048):
            z = torch.mm(wt, st["x"][i:i + 2048].double().t().contiguous()).t() + st["bias"].double()
            y = _curve(z, c["act"])
            ys.append(y if st["res"] is None else y + st["res"][i:i + 2048].double())
            zs.append(z)
        return torch.cat(ys) if st["z"] is None else (torch.cat(ys), torch.cat(zs))
    dz, db = [], torch.zeros(M, dtype=torch.float64, device=DEV)
    for i in range(0, N, 1024):
        z = st["z"][i:i + 1024].double().requires_grad_()
        _curve(z, c["act"]).backward(st["dy"][i:i + 1024].double())
        dz.append(z.grad)
        db += z.grad.sum(0)
    return torch.cat(dz), db


def _exact_balance(st, c):
    """Sequence by sequence; the gradient from autograd of the two functions of the logits."""
    N, E, k, T = c["N"], c["E"], c["k"], c["T"]
    S = (N + T - 1) // T
    if S > 2000:
        return None
    s = st["scores"].double()
    keep = torch.ones(N, dtype=torch.bool, device=DEV) if st["mask"] is None else st["mask"] != 0
    if c["dir"] == "fwd":
        counts = torch.zeros((S, E), dtype=torch.int32, device=DEV)
        coef = torch.zeros((S, E), dtype=torch.float64, device=DEV)
        loss = torch.zeros(1, dtype=torch.float64, device=DEV)
        for q in range(S):
            rows = keep[q * T:(q + 1) * T]
            mine = s[q * T:(q + 1) * T][rows]
            V = mine.shape[0]
            if V == 0:
                continue
            n = torch.bincount(st["idx"][q * T:(q + 1) * T][rows].long().reshape(-1), minlength=E)
            counts[q] = n.to(torch.int32)
            share = n.double() / (k * V) * E
            loss += st["weight"] / S * torch.dot(share, torch.nn.functional.normalize(mine, p=1.0, dim=1).mean(0))
            coef[q] = st["weight"] / S * share / V
        return loss, counts, coef
    s.requires_grad_()
    i = st["idx"].long()
    picked = torch.gather(s, 1, i)
    weights = st["alpha"] * picked / (picked.sum(1, keepdim=True) + 1e-20)
    prob = torch.nn.functional.normalize(s, p=1.0, dim=1)
    rows = torch.div(torch.arange(N, device=DEV), T, rounding_mode="floor")
    balance = (prob * st["coef"].double().index_select(0, rows)).sum(1)
    ((weights * st["dw"].double()).sum() + st["dloss"].double().sum() * balance[keep].sum()).backward()
    with torch.no_grad():
        return s.grad * (s - s * s)


def _exact_clip(st, c):
    norm = torch.linalg.vector_norm(torch.cat([g.double() for g in st["grads"]])).view(1)
    factor = min(1.0, st["max"] / (float(norm) + 1e-6))
    return [norm] + [g.double() * factor for g in st["grads"]]
