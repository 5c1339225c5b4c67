"""Timing cases of the operators around the experts: block norms, grouped products, combine, 4-bit products.

  norm      h_out = a h + gate * (o / rms(o)) w_post and u = (h_out / rms(h_out)) w_pre in one pass, and
            its backward pass
  combine   y[n] = alpha sum_s w[n, s] rows[inv[n, s]] + shared[n], and its backward pass
  grouped   y[r] = W[e(r)] x[src(r)] over rows grouped by expert, the gradients of x and of W
  quant     the same product with 4-bit weights and one scale per group of a row, optionally with the
            SwiGLU of its two halves

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


def listed():
    return [
        # One token of a GLM-5-wide decoder between two blocks: closes one block, opens the next. Latency.
        {"name": "norm_step", "op": "norm", "dir": "fwd", "N": 1, "D": 6144, "dtype": "bf16", "gate": "channel"},
        # A prompt of 8,191 tokens of the GLM-4.5 width between two blocks, no gate.
        {"name": "norm_prefill", "op": "norm", "dir": "fwd", "N": 8191, "D": 5120, "dtype": "bf16", "gate": "none"},
        # Training step of the Air width: eight sequences of 512 tokens, one gate row per sequence.
        {"name": "norm_backward", "op": "norm", "dir": "bwd", "N": 4096, "D": 4096, "dtype": "bf16", "gate": "seq512"},
        # Weighted sum of the experts' rows in a float32 evaluation of 1,000 tokens.
        {"name": "combine_f32", "op": "combine", "dir": "fwd", "N": 1000, "D": 4096, "k": 8, "dtype": "f32"},
        # Gradients of the experts' rows and of the mixture weights, Air width.
        {"name": "combine_backward", "op": "combine", "dir": "bwd", "N": 4096, "D": 4096, "k": 8, "dtype": "bf16"},
        # Down projection of a decode batch of 32 requests over GLM-5's 256 experts: a weight stream.
        {"name": "grouped_decode", "op": "grouped", "dir": "fwd", "N": 32, "k": 8, "E": 256, "K": 2048, "M": 6144,
         "gather": False, "dtype": "bf16"},
        # Gate and up projection of an Air-shaped prompt, tokens gathered by the dispatch lists.
        {"name": "grouped_prefill", "op": "grouped", "dir": "fwd", "N": 4096, "k": 8, "E": 128, "K": 4096, "M": 2816,
         "gather": True, "dtype": "bf16"},
        # Input gradient of the GLM-4.5 down projection, 3,001 tokens.
        {"name": "grouped_dgrad", "op": "grouped", "dir": "dgrad", "N": 3001, "k": 8, "E": 160, "K": 1536, "M": 5120,
         "gather": False, "dtype": "bf16"},
        # Weight gradient of the Air gate and up projection.
        {"name": "grouped_wgrad", "op": "grouped", "dir": "wgrad", "N": 4096, "k": 8, "E": 128, "K": 4096, "M": 2816,
         "gather": True, "dtype": "bf16"},
        # One token through the 4-bit gate and up projection of the GLM-4.5 dense layers.
        {"name": "quant_token", "op": "quant", "N": 1, "k": 1, "E": 1, "K": 5120, "M": 24576, "group": 128,
         "swiglu": True},
        # A decode batch of 32 requests through GLM-5's experts in 4 bits, groups of 32.
        {"name": "quant_decode", "op": "quant", "N": 32, "k": 8, "E": 256, "K": 6144, "M": 4096, "group": 32,
         "swiglu": True},
        # A ragged prompt through the 4-bit down projection of the GLM-4.5 dense layers.
        {"name": "quant_prompt", "op": "quant", "N": 1021, "k": 1, "E": 1, "K": 12288, "M": 5120, "group": 64,
         "swiglu": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _wide(rng, lo, hi):
    """A multiple of 64 between lo and hi, spread over the logarithm."""
    return max(1, int(round(_log(rng, lo, hi) / 64))) * 64


def draw(rng):
    op = rng.choice(["norm", "norm", "combine", "grouped", "grouped", "grouped", "quant", "quant"])
    if op == "norm":
        c = {"op": op, "dir": rng.choice(["fwd", "bwd"]), "N": _log(rng, 1, 8192), "D": _wide(rng, 256, 6144),
             "dtype": rng.choice(["bf16", "bf16", "f32"]), "gate": rng.choice(["none", "channel", "token", "seq512"])}
        while c["N"] * c["D"] > (1 << 24) * (2 if c["dtype"] == "bf16" and c["dir"] == "fwd" else 1):
            c["N"] = c["N"] * 2 // 3
        return c
    if op == "combine":
        c = {"op": op, "dir": rng.choice(["fwd", "bwd"]), "N": _log(rng, 1, 4096), "D": _wide(rng, 256, 6144),
             "k": rng.choice([1, 2, 4, 6, 8]), "dtype": rng.choice(["bf16", "bf16", "f32"])}
        while c["N"] * c["D"] * c["k"] > (1 << 27) // (1 if c["dtype"] == "bf16" else 2):
            c["N"] = c["N"] * 2 // 3
        return c
    if op == "grouped":
        f32 = rng.random() < 0.2
        c = {"op": op, "dir": rng.choice(["fwd", "dgrad", "wgrad"]), "N": _log(rng, 1, 4096),
             "k": rng.choice([1, 2, 4, 8]), "E": rng.choice([8, 16, 60, 128, 160, 256]),
             "K": _wide(rng, 256, 6144 if not f32 else 1536), "M": _wide(rng, 256, 6144 if not f32 else 1536),
             "gather": rng.random() < 0.5, "dtype": "f32" if f32 else "bf16"}
        if c["dir"] == "dgrad":
            c["gather"] = False
        c["k"] = min(c["k"], c["E"])
        while c["E"] * c["K"] * c["M"] > 1500000000 // (8 if f32 else 1):
            c["E"] = max(1, c["E"] // 2)
            c["k"] = min(c["k"], c["E"])
        while c["N"] * c["k"] * c["K"] * c["M"] > 370000000000 // (64 if f32 else 1):
            c["N"] = c["N"] * 2 // 3
        return c
    c = {"op": "quant", "N": _log(rng, 1, 1024), "k": 1, "E": 1, "K": 0, "M": _wide(rng, 256, 16384),
         "group": rng.choice([32, 64, 128]), "swiglu": rng.random() < 0.5}
    c["K"] = max(1, int(round(_log(rng, 256, 12288) / 128))) * 128
    if c["swiglu"]:
        c["M"] = max(128, c["M"] // 128 * 128)
    if rng.random() < 0.5:
        c["E"] = rng.choice([8, 60, 128, 160, 256])
        c["k"] = rng.choice([1, 2, 4, 8])
        while c["E"] * c["K"] * c["M"] > 6400000000:
            c["E"] //= 2
        c["k"] = min(c["k"], c["E"])
    while c["N"] * c["k"] * c["K"] * c["M"] > 64000000000:
        c["N"] = c["N"] * 2 // 3
    return c


# ---- inputs ----
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _randn(g, shape, dtype, std=1.0):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).mul_(std).to(dtype)


def _weights(g, E, M, K, dtype):
    """[E, M, K] of variance 1 / K, one expert at a time (the float32 draw of all of them is large)."""
    w = torch.empty((E, M, K), dtype=dtype, device=DEV)
    for e in range(E):
        w[e] = _randn(g, (M, K), dtype, 1.0 / math.sqrt(K))
    return w


def _gate_rows(case):
    """Rows that share one gate row: all of them, one, or a sequence's."""
    if case["gate"] == "seq512":
        return 512
    return 1 if case["gate"] == "token" else max(1, case["N"])


def _routing(g, N, k, E):
    """Lists of a random uneven routing: offsets [E + 1], sorted_pair [N k], inv_row [N k], counts on the host."""
    logits = torch.randn((N, E), generator=g, device=DEV) + 0.3 * torch.randn((1, E), generator=g, device=DEV)
    flat = logits.topk(k, dim=1).indices.reshape(-1)
    order = torch.sort(flat, stable=True).indices
    counts = torch.bincount(flat, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = torch.cumsum(counts, 0).to(torch.int32)
    inv = torch.empty_like(order)
    inv[order] = torch.arange(N * k, device=DEV)
    return offsets, order.to(torch.int32), inv.to(torch.int32), counts.tolist()


def prepare(case, seed):
    g = _gen(seed)
    st = {"case": dict(case)}
    op = case["op"]
    if op == "norm":
        N, D, dt = case["N"], case["D"], TYPES[case["dtype"]]
        st["T"] = _gate_rows(case)
        G = (N + st["T"] - 1) // st["T"]
        st["a"] = 0.9
        st["h"] = _randn(g, (N, D), dt, 2.0)
        st["o"] = _randn(g, (N, D), dt, 0.5)
        st["w_post"] = (1.0 + 0.1 * torch.randn(D, generator=g, device=DEV)).to(dt)
        st["w_pre"] = (1.0 + 0.1 * torch.randn(D, generator=g, device=DEV)).to(dt)
        st["gate"] = None
        if case["gate"] != "none":
            st["gate"] = (0.5 + 0.2 * torch.randn((G, D), generator=g, device=DEV)).to(dt)
        if case["dir"] == "fwd":
            st["out"] = (torch.empty_like(st["h"]), torch.empty_like(st["h"]))
        else:
            st["d_h_out"] = _randn(g, (N, D), dt)
            st["d_u"] = _randn(g, (N, D), dt)
            f = {"dtype": torch.float32, "device": DEV}
            st["out"] = (torch.empty_like(st["h"]), torch.empty_like(st["h"]), torch.empty(D, **f),
                         None if st["gate"] is None else torch.empty((G, D), **f), torch.empty(D, **f))
            if own:
                import sparse_moe_layer_gate_amd as moe

                n = moe.moe_block_norm_workspace_size(N, D, case["dtype"], st["T"])
                st["ws"] = torch.empty(max(n, 256), dtype=torch.uint8, device=DEV)
    elif op == "combine":
        N, D, k, dt = case["N"], case["D"], case["k"], TYPES[case["dtype"]]
        _, _, st["inv"], _ = _routing(g, N, k, 128)
        st["rows"] = _randn(g, (N * k, D), dt)
        w = torch.rand((N, k), generator=g, device=DEV) + 0.1
        st["w"] = (w / w.sum(1, keepdim=True)).contiguous()
        st["alpha"] = 2.5
        if case["dir"] == "fwd":
            st["shared"] = _randn(g, (N, D), dt)
            st["out"] = torch.empty((N, D), dtype=dt, device=DEV)
        else:
            st["dy"] = _randn(g, (N, D), dt)
            st["out"] = (torch.empty_like(st["rows"]), torch.empty_like(st["w"]))
    elif op == "grouped":
        N, k, E, K, M, dt = case["N"], case["k"], case["E"], case["K"], case["M"], TYPES[case["dtype"]]
        R = N * k
        st["offsets"], st["pair"], _, st["counts"] = _routing(g, N, k, E)
        if case["dir"] != "dgrad":
            st["x"] = _randn(g, (N if case["gather"] else R, K), dt)
        if case["dir"] != "fwd":
            st["dy"] = _randn(g, (R, M), dt)
        if case["dir"] != "wgrad":
            st["w"] = _weights(g, E, M, K, dt)
        shape = {"fwd": (R, M), "dgrad": (R, K), "wgrad": (E, M, K)}[case["dir"]]
        st["out"] = torch.empty(shape, dtype=dt, device=DEV)
        if own:
            import sparse_moe_layer_gate_amd as moe

            n = moe.moe_grouped_workspace_size(E, R, case["dtype"])
            st["ws"] = torch.empty(max(n, 256), dtype=torch.uint8, device=DEV)
    else:
        N, k, E, K, M, group = case["N"], case["k"], case["E"], case["K"], case["M"], case["group"]
        if E > 1:
            st["offsets"], st["pair"], _, st["counts"] = _routing(g, N, k, E)
        else:
            st["offsets"], st["pair"], st["counts"] = None, None, [N]
        st["x"] = _randn(g, (N, K), torch.bfloat16)
        st["q"] = torch.empty((E, M, K // 2), dtype=torch.uint8, device=DEV)
        st["s"] = torch.empty((E, M, K // group), dtype=torch.bfloat16, device=DEV)
        for e in range(E):
            w = torch.randn((M, K // group, group), generator=g, device=DEV).mul_(1.0 / math.sqrt(K))
            s = (w.abs().amax(2) / 7.0).to(torch.bfloat16)
            q = (torch.round(w / s.float()[..., None]).clamp_(-8, 7) + 8).to(torch.uint8).reshape(M, K // 2, 2)
            st["q"][e] = q[..., 0] | (q[..., 1] << 4)
            st["s"][e] = s
        st["out"] = torch.empty((N * k, M // 2 if case["swiglu"] else M), dtype=torch.bfloat16, device=DEV)
    return st


# ---- one pass ----
def run(st):
    c = st["case"]
    return globals()[("_own_" if own else "_plain_") + c["op"]](st, c)


def _own_norm(st, c):
    import sparse_moe_layer_gate_amd as moe

    if c["dir"] == "fwd":
        h_out, u = st["out"]
        moe.moe_block_norm(c["N"], st["h"], st["o"], st["w_post"], st["gate"], st["T"], st["w_pre"], h_out, u,
                           residual_scale=st["a"], eps=EPS)
        return h_out, u
    dh, do, dw_post, dgate, dw_pre = st["out"]
    moe.moe_block_norm_backward(c["N"], st["h"], st["o"], st["w_post"], st["gate"], st["T"], st["w_pre"],
                                st["d_h_out"], st["d_u"], dh, do, dw_post, dgate, dw_pre, st["ws"],
                                residual_scale=st["a"], eps=EPS)
    return tuple(t for t in st["out"] if t is not None)


def _own_combine(st, c):
    import sparse_moe_layer_gate_amd as moe

    if c["dir"] == "fwd":
        moe.moe_combine(c["N"], c["k"], st["rows"], st["inv"], st["w"], st["shared"], st["out"], alpha=st["alpha"])
        return st["out"]
    drows, dw = st["out"]
    moe.moe_combine_backward(c["N"], c["k"], st["dy"], st["rows"], st["inv"], st["w"], drows, dw, alpha=st["alpha"])
    return drows, dw


def _own_grouped(st, c):
    import sparse_moe_layer_gate_amd as moe

    index, div = (st["pair"], c["k"]) if c["gather"] else (None, 1)
    if c["dir"] == "fwd":
        moe.moe_grouped_linear(st["x"], st["w"], st["offsets"], st["out"], st["ws"], row_index=index, index_div=div)
    elif c["dir"] == "dgrad":
        moe.moe_grouped_linear_dgrad(st["dy"], st["w"], st["offsets"], st["out"], st["ws"])
    else:
        moe.moe_grouped_linear_wgrad(st["dy"], st["x"], st["offsets"], st["out"], st["ws"], row_index=index,
                                     index_div=div)
    return st["out"]


def _own_quant(st, c):
    import sparse_moe_layer_gate_amd as moe

    moe.moe_qlinear(st["x"], st["q"], st["s"], st["out"], offsets=st["offsets"], row_index=st["pair"],
                    index_div=c["k"], swiglu=c["swiglu"])
    return st["out"]


def _gate_of(st, N):
    """The gate of every row in float32, or 1."""
    if st["gate"] is None:
        return 1.0
    return st["gate"].float()[torch.arange(N, device=DEV) // st["T"]]


def _plain_norm(st, c):
    dt = TYPES[c["dtype"]]
    h, o = st["h"].float(), st["o"].float()
    w_post, w_pre, gate = st["w_post"].float(), st["w_pre"].float(), _gate_of(st, c["N"])
    on = o * torch.rsqrt((o * o).mean(1, keepdim=True) + EPS)
    if c["dir"] == "fwd":
        h_out = st["a"] * h + gate * (on * w_post)
        u = h_out * torch.rsqrt((h_out * h_out).mean(1, keepdim=True) + EPS) * w_pre
        return h_out.to(dt), u.to(dt)
    # backward: h is the block's output, from which the norm before the next block started
    r = torch.rsqrt((h * h).mean(1, keepdim=True) + EPS)
    hn = h * r
    du = st["d_u"].float()
    t = du * w_pre
    d = st["d_h_out"].float() + r * (t - hn * (t * hn).mean(1, keepdim=True))
    dw_pre = (du * hn).sum(0)
    dn = d * gate
    dw_post = (dn * on).sum(0)
    t = dn * w_post
    ro = torch.rsqrt((o * o).mean(1, keepdim=True) + EPS)
    do = ro * (t - on * (t * on).mean(1, keepdim=True))
    out = [(st["a"] * d).to(dt), do.to(dt), dw_post]
    if st["gate"] is not None:
        dgate = torch.zeros(st["gate"].shape, dtype=torch.float32, device=DEV)
        T = st["T"]
        for i in range(dgate.shape[0]) if T > 1 else ():
            dgate[i] = (d[i * T:(i + 1) * T] * on[i * T:(i + 1) * T] * w_post).sum(0)
        if T == 1:
            dgate = d * on * w_post
        out.append(dgate)
    out.append(dw_pre)
    return tuple(out)


def _plain_combine(st, c):
    dt = TYPES[c["dtype"]]
    N, k = c["N"], c["k"]
    inv = st["inv"].long().view(N, k)
    if c["dir"] == "fwd":
        acc = torch.zeros((N, c["D"]), dtype=torch.float32, device=DEV)
        for s in range(k):
            acc += st["w"][:, s:s + 1] * st["rows"][inv[:, s]].float()
        return (st["alpha"] * acc + st["shared"].float()).to(dt)
    dy = st["dy"].float() * st["alpha"]
    drows = torch.empty_like(st["rows"])
    dw = torch.empty_like(st["w"])
    for s in range(k):
        drows[inv[:, s]] = (st["w"][:, s:s + 1] * dy).to(dt)
        dw[:, s] = (dy * st["rows"][inv[:, s]].float()).sum(1)
    return drows, dw


def _source(st, c):
    """The row of x behind every grouped row."""
    if st.get("pair") is not None and c.get("gather", True):
        return st["pair"].long() // c["k"]
    return torch.arange(c["N"] * c["k"], device=DEV)


def _plain_grouped(st, c):
    dt = TYPES[c["dtype"]]
    src = _source(st, c)
    shape = {"fwd": (c["N"] * c["k"], c["M"]), "dgrad": (c["N"] * c["k"], c["K"]),
             "wgrad": (c["E"], c["M"], c["K"])}[c["dir"]]
    out = torch.empty(shape, dtype=dt, device=DEV)
    a = 0
    for e, n in enumerate(st["counts"]):
        b = a + n
        if c["dir"] == "wgrad":
            if n:
                out[e] = st["dy"][a:b].float().t().mm(st["x"][src[a:b]].float()).to(dt)
            else:
                out[e].zero_()
        elif n:
            if c["dir"] == "fwd":
                out[a:b] = st["x"][src[a:b]].float().mm(st["w"][e].float().t()).to(dt)
            else:
                out[a:b] = st["dy"][a:b].float().mm(st["w"][e].float()).to(dt)
        a = b
    return out


def _dequantize(q, s, dtype):
    """[M, K / 2] nibbles (even k low) and [M, K / group] scales -> [M, K]."""
    M, half = q.shape
    v = torch.stack((q & 15, q >> 4), 2).reshape(M, 2 * half).to(dtype) - 8.0
    return (v.view(M, s.shape[1], -1) * s.to(dtype)[..., None]).view(M, 2 * half)


def _plain_quant(st, c):
    src = _source(st, c)
    out = torch.empty_like(st["out"])
    a = 0
    for e, n in enumerate(st["counts"]):
        b = a + n
        if n:
            y = st["x"][src[a:b]].float().mm(_dequantize(st["q"][e], st["s"][e], torch.float32).t())
            if c["swiglu"]:
                g, u = y[:, :c["M"] // 2], y[:, c["M"] // 2:]
                y = g / (1.0 + torch.exp(-g)) * u
            out[a:b] = y.to(torch.bfloat16)
        a = b
    return out


# ---- what a pass cannot do without ----
def _experts_used(c):
    """Experts with at least one of the batch's tokens, expected under even routing."""
    return c["E"] * (1.0 - (1.0 - min(1.0, c["k"] / c["E"])) ** c["N"]) if c["E"] > 1 else 1.0


def work(c):
    if c["op"] == "norm":
        es = 4 if c["dtype"] == "f32" else 2
        N, D, T = c["N"], c["D"], _gate_rows(c)
        gate = 0 if c["gate"] == "none" else (N + T - 1) // T * D
        if c["dir"] == "fwd":
            return {"bytes": es * (4 * N * D + 2 * D + gate), "flops": 12 * N * D}
        return {"bytes": es * (6 * N * D + 2 * D + gate) + 4 * (2 * D + gate), "flops": 30 * N * D}
    if c["op"] == "combine":
        es = 4 if c["dtype"] == "f32" else 2
        N, D, k = c["N"], c["D"], c["k"]
        if c["dir"] == "fwd":
            return {"bytes": es * N * D * (k + 2) + 8 * N * k, "flops": 2 * N * D * (k + 1)}
        return {"bytes": es * N * D * (2 * k + 1) + 12 * N * k, "flops": 3 * N * D * k}
    R = c["N"] * c["k"]
    if c["op"] == "grouped":
        es = 4 if c["dtype"] == "f32" else 2
        x = (c["N"] if c["gather"] else R) * c["K"]
        w = (c["E"] if c["dir"] == "wgrad" else _experts_used(c)) * c["K"] * c["M"]
        return {"bytes": int(es * (x + R * c["M"] + w)), "flops": 2 * R * c["K"] * c["M"]}
    w = _experts_used(c) * c["M"] * (c["K"] / 2 + 2 * c["K"] / c["group"])
    y = R * (c["M"] // 2 if c["swiglu"] else c["M"])
    return {"bytes": int(w + 2 * (c["N"] * c["K"] + y)), "flops": 2 * R * c["K"] * c["M"]}


# ---- the definitions in float64 ----
def exact(case, seed):
    st = prepare(case, seed)
    c = case
    if c["op"] == "norm":
        return _exact_norm(st, c)
    if c["op"] == "combine":
        return _exact_combine(st, c)
    if c["op"] == "grouped":
        return _exact_grouped(st, c)
    return _exact_quant(st, c)


def _exact_norm(st, c):
    """Row blocks of the formulas; the gradients from autograd of the forward formula."""
    N, D = c["N"], c["D"]
    p = {n: None if st[n] is None else st[n].double() for n in ("w_post", "w_pre", "gate")}

    def rms(v):
        return v / torch.sqrt(v.square().sum(-1, keepdim=True) / D + EPS)

    def expand(gate, i, j):
        return 1.0 if gate is None else gate.index_select(0, torch.arange(i, j, device=DEV).div(st["T"],
                                                                                               rounding_mode="floor"))
    if c["dir"] == "fwd":
        h_out, u = [], []
        for i in range(0, N, 1024):
            j = min(N, i + 1024)
            v = st["a"] * st["h"][i:j].double() + expand(p["gate"], i, j) * rms(st["o"][i:j].double()) * p["w_post"]
            h_out.append(v)
            u.append(rms(v) * p["w_pre"])
        return torch.cat(h_out), torch.cat(u)
    leaves = {n: v.requires_grad_() for n, v in p.items() if v is not None}
    dh, do = [], []
    for i in range(0, N, 1024):
        j = min(N, i + 1024)
        # d u / d h_out at the given h_out, then the rest of the pass at h_out's whole gradient
        h = st["h"][i:j].double().requires_grad_()
        (rms(h) * leaves["w_pre"]).backward(st["d_u"][i:j].double())
        d = st["d_h_out"][i:j].double() + h.grad
        o = st["o"][i:j].double().requires_grad_()
        (expand(leaves.get("gate"), i, j) * (rms(o) * leaves["w_post"])).backward(d)
        dh.append(st["a"] * d)
        do.append(o.grad)
    out = [torch.cat(dh), torch.cat(do), leaves["w_post"].grad]
    if "gate" in leaves:
        out.append(leaves["gate"].grad)
    out.append(leaves["w_pre"].grad)
    return tuple(out)


def _exact_combine(st, c):
    N, k = c["N"], c["k"]
    inv = st["inv"].long()
    w = st["w"].double()
    if c["dir"] == "fwd":
        y = st["shared"].double()
        token = torch.arange(N * k, device=DEV) // k
        step = max(k, (1 << 25) // c["D"] // k * k)
        for i in range(0, N * k, step):
            part = st["rows"].index_select(0, inv[i:i + step]).double() * (st["alpha"] * w.view(-1)[i:i + step, None])
            n0, n1 = int(i // k), min(N, (i + step) // k)
            y[n0:n1] += part.view(n1 - n0, k, c["D"]).sum(1)
        del token
        return y
    pair = torch.empty_like(inv)
    pair[inv] = torch.arange(N * k, device=DEV)
    drows = torch.empty(st["rows"].shape, dtype=torch.float64, device=DEV)
    dot = torch.empty(N * k, dtype=torch.float64, device=DEV)
    for i in range(0, N * k, 4096):
        p = pair[i:i + 4096]
        g = st["alpha"] * st["dy"].index_select(0, p // k).double()
        drows[i:i + 4096] = w.view(-1)[p][:, None] * g
        dot[p] = (g * st["rows"][i:i + 4096].double()).sum(1)
    return drows, dot.view(N, k)


def _exact_grouped(st, c):
    R, E = c["N"] * c["k"], c["E"]
    rows = torch.arange(R, device=DEV)
    expert = torch.searchsorted(st["offsets"].long()[1:].contiguous(), rows, right=True)
    src = torch.div(st["pair"].long(), c["k"], rounding_mode="floor") if c["gather"] else rows
    shape = {"fwd": (R, c["M"]), "dgrad": (R, c["K"]), "wgrad": (E, c["M"], c["K"])}[c["dir"]]
    out = torch.zeros(shape, dtype=torch.float64, device=DEV)
    for e in torch.unique(expert).tolist():
        sel = torch.nonzero(expert == e).view(-1)
        if c["dir"] == "fwd":
            out[sel] = torch.mm(st["w"][e].double(), st["x"][src[sel]].double().t().contiguous()).t()
        elif c["dir"] == "dgrad":
            out[sel] = torch.mm(st["w"][e].double().t().contiguous(), st["dy"][sel].double().t().contiguous()).t()
        else:
            out[e] = torch.mm(st["x"][src[sel]].double().t().contiguous(), st["dy"][sel].double()).t()
    return out


def _exact_quant(st, c):
    R, half = c["N"] * c["k"], c["M"] // 2
    if st["offsets"] is None:
        bounds, src = [0, R], torch.arange(R, device=DEV)
    else:
        bounds, src = st["offsets"].tolist(), torch.div(st["pair"].long(), c["k"], rounding_mode="floor")
    out = torch.empty((R, half if c["swiglu"] else c["M"]), dtype=torch.float64, device=DEV)
    for e in range(c["E"]):
        a, b = bounds[e], bounds[e + 1]
        if a == b:
            continue
        w = torch.empty((c["M"], c["K"]), dtype=torch.float64, device=DEV)
        w[:, 0::2] = torch.bitwise_and(st["q"][e], 15).double()
        w[:, 1::2] = torch.bitwise_right_shift(st["q"][e], 4).double()
        w.sub_(8.0).mul_(st["s"][e].double().repeat_interleave(c["group"], 1))
        y = torch.mm(w, st["x"][src[a:b]].double().t().contiguous()).t()
        if c["swiglu"]:
            y = y[:, :half] * torch.sigmoid(y[:, :half]) * y[:, half:]
        out[a:b] = y
    return out
