"""Plain float64 references of the operators around the experts, with bounds on what float32 arithmetic may
differ by, for the tests. Everything here runs on the CPU in numpy / torch float64.

Bounds count rounding steps: a value stored in bfloat16 is off by at most 2^-8 of itself and one in float32
by 2^-24; a float32 sum of n terms by at most n 2^-24 times the sum of the terms' magnitudes, whatever the
order. Integer-valued inputs whose sums stay below 2^24 leave no float32 error at all, so products of them
have to equal the once-rounded exact value bit for bit.
"""
import torch

U32 = 2.0 ** -24
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: U32}


def ints(g, shape, lo, hi, dtype=torch.bfloat16):
    return torch.randint(lo, hi + 1, shape, generator=g).to(dtype)


def lists(g, N, k, E, empty=0.0):
    """Routing of N tokens: distinct experts per token, a share of the slots empty (id E). Returns topk [N, k]
    int32, offsets [E + 1], sorted_pair [N k] (rows in use first), inv_row [N k] (-1: empty)."""
    topk = torch.rand((N, E), generator=g).topk(k, 1).indices.to(torch.int32)
    if empty:
        topk[torch.rand((N, k), generator=g) < empty] = E
    flat = topk.reshape(-1).long()
    order = torch.sort(flat, stable=True).indices
    used = int((flat < E).sum())
    counts = torch.bincount(flat, minlength=E + 1)[:E]
    offsets = torch.zeros(E + 1, dtype=torch.int32)
    offsets[1:] = counts.cumsum(0)
    inv = torch.full((N * k,), -1, dtype=torch.int32)
    inv[order[:used]] = torch.arange(used, dtype=torch.int32)
    pair = torch.zeros(N * k, dtype=torch.int32)
    pair[:used] = order[:used].to(torch.int32)
    return topk, offsets, pair, inv


def expert_of(offsets):
    o = offsets.tolist()
    return [(e, o[e], o[e + 1]) for e in range(len(o) - 1) if o[e + 1] > o[e]]


# ---- block norm ----
def norm_forward(h, o, w_post, gate, T, w_pre, a, eps):
    """(h_out, u) in float64; absent parts are None."""
    N, D = h.shape
    v = h
    if o is not None:
        m = o
        if w_post is not None:
            m = o / torch.sqrt(o.square().mean(1, keepdim=True) + eps) * w_post
        if gate is not None:
            m = m * gate[torch.arange(N) // T]
        v = a * h + m
    u = None
    if w_pre is not None:
        u = v / torch.sqrt(v.square().mean(1, keepdim=True) + eps) * w_pre
    return v, u


def norm_forward_bound(h, o, w_post, gate, T, w_pre, a, eps):
    """Largest float32 errors of (h_out, u): c of the magnitudes that a row's values are made of, with c for the
    D-term sum behind a norm (halved by the square root) and a dozen further steps."""
    D = h.shape[1]
    c = (D / 2 + 16) * U32
    v, u = norm_forward(h, o, w_post, gate, T, w_pre, a, eps)
    if o is None:
        mag = torch.zeros_like(v)
    else:
        mag = (a * h).abs() + (v - a * h).abs()
    ev = c * mag
    if u is None:
        return ev, None
    r = w_pre.abs() / torch.sqrt(v.square().mean(1, keepdim=True) + eps)
    eu = c * u.abs() + r * ev + u.abs() * ev.norm(dim=1, keepdim=True) / v.norm(dim=1, keepdim=True).clamp_min(1e-300)
    return ev, eu


def norm_backward(h, o, w_post, gate, T, w_pre, dv, du, a, eps):
    """Gradients (dh, do, dw_post, dgate, dw_pre) in float64 by the formulas, and their float32 error bounds: the
    same formulas over magnitudes, times the steps behind a value (two D-term sums, and for the parameter
    gradients the sum over N rows)."""
    out = []
    for mag in (False, True):
        ab = (lambda t: t.abs()) if mag else (lambda t: t)
        sub = (lambda p, q: p + q) if mag else (lambda p, q: p - q)
        d = torch.zeros_like(h if h is not None else o) if dv is None else ab(dv)
        dw_pre = None
        if w_pre is not None:
            r = 1.0 / torch.sqrt(h.square().mean(1, keepdim=True) + eps)
            n, t = ab(h * r), ab(du) * ab(w_pre)
            d = d + r * sub(t, n * (t * n).mean(1, keepdim=True))
            dw_pre = (ab(du) * n).sum(0)
        if o is None:
            out.append((d, None, None, None, dw_pre))
            continue
        ro = torch.ones_like(o[:, :1])
        if w_post is not None:
            ro = 1.0 / torch.sqrt(o.square().mean(1, keepdim=True) + eps)
        m = ab(o * ro)
        wp = ab(w_post) if w_post is not None else 1.0
        g = ab(gate[torch.arange(o.shape[0]) // T]) if gate is not None else 1.0
        z = d * g * wp
        do = ro * sub(z, m * (z * m).mean(1, keepdim=True)) if w_post is not None else z
        dgate = None
        if gate is not None:
            dgate = torch.zeros_like(gate).index_add(0, torch.arange(o.shape[0]) // T, d * m * wp)
        out.append((abs(a) * d if mag else a * d, do, (d * g * m).sum(0) if w_post is not None else None, dgate, dw_pre))
    N, D = (o if o is not None else h).shape
    c = (2 * D + 40) * U32
    cs = [c, c, c + N * U32, c + N * U32, c + N * U32]
    return out[0], [None if b is None else k * b for k, b in zip(cs, out[1])]


# ---- combine ----
def combine(rows, inv, w, shared, alpha, N, k):
    y = torch.zeros((N, rows.shape[1]), dtype=torch.float64)
    mag = y.clone()
    for s in range(k):
        r = inv.view(N, k)[:, s].long()
        ok = (r >= 0) & (r < rows.shape[0])
        part = rows[r.clamp(0, max(rows.shape[0] - 1, 0))] * (1.0 if w is None else w[:, s:s + 1])
        y += torch.where(ok[:, None], part, torch.zeros_like(part))
        mag += torch.where(ok[:, None], part.abs(), torch.zeros_like(part))
    y, mag = alpha * y, abs(alpha) * mag
    if shared is not None:
        y, mag = y + shared, mag + shared.abs()
    return y, (k + 3) * U32 * mag


# ---- grouped products ----
def grouped(x, w, offsets, src, R):
    y = torch.zeros((R, w.shape[1]), dtype=torch.float64)
    for e, a, b in expert_of(offsets):
        y[a:b] = x[src[a:b]] @ w[e].t()
    return y


def grouped_dgrad(dy, w, offsets):
    dx = torch.zeros((dy.shape[0], w.shape[2]), dtype=torch.float64)
    for e, a, b in expert_of(offsets):
        dx[a:b] = dy[a:b] @ w[e]
    return dx


def grouped_wgrad(dy, x, offsets, src, E):
    dw = torch.zeros((E, dy.shape[1], x.shape[1]), dtype=torch.float64)
    for e, a, b in expert_of(offsets):
        dw[e] = dy[a:b].t() @ x[src[a:b]]
    return dw


# ---- 4-bit weights ----
def dequantize(q, s):
    E, M, half = q.shape
    v = torch.empty((E, M, 2 * half), dtype=torch.float64)
    v[..., 0::2] = (q & 15).double() - 8
    v[..., 1::2] = (q >> 4).double() - 8
    return v * s.double().repeat_interleave(2 * half // s.shape[2], 2)


def check(name, got, ref, bound):
    """Every element within its float32 bound and half a step of its type."""
    got = got.detach().cpu()
    r = ref.double()
    err = (got.double() - r).abs()
    tol = bound + HALF_STEP[got.dtype] * (r.abs() + bound) + 1e-37
    worst = float((err / tol).max()) if err.numel() else 0.0
    print(f"  {name}: worst error / tolerance {worst:.3g}", flush=True)
    assert torch.isfinite(got.double()).all() and worst <= 1.0, (name, worst)
