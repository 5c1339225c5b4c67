"""Plain float64 references of the operators of a training step, with bounds on what float32 arithmetic may differ by,
for the tests. Everything here runs on the CPU in torch float64.

Bounds count rounding steps of U = 2^-24 each. A sum over the features of a row passes each term through at most 8 x 4
additions in a thread, 6 in a wave and 16 over the waves: fewer than SUM = 64. Activations of results rounded to
bfloat16 may be off by 2^-13 of themselves (a hardware exponential and reciprocal, a polynomial of relative error
4e-5); float32 ones by a few steps and by what the rounding of the exponent's argument, of size about z^2, makes of it.
"""
import math

import torch

from tests._ops import HALF_STEP, U32 as U

SUM = 64


# ---- layer norm ----
def layer_norm(x, residual, w, b, eps):
    """(h, y, stats) and their bounds; h is None without a residual."""
    h = x if residual is None else x + residual
    mean = h.mean(1, keepdim=True)
    d = h - mean
    r = 1.0 / torch.sqrt(d.square().mean(1, keepdim=True) + eps)
    w = torch.ones(h.shape[1], dtype=h.dtype) if w is None else w
    b = torch.zeros_like(w) if b is None else b
    y = d * r * w + b
    rms, ad = h.square().mean(1, keepdim=True).sqrt(), d.abs().mean(1, keepdim=True)
    # the centred value: sums of what is left around a first mean, and h's own rounding
    ey = (SUM + 36) * U * w.abs() * r * (d.abs() + ad) + 2 * U * w.abs() * r * (h.abs() + d.abs() * rms * r)
    ey = ey + 2 * U * (y.abs() + b.abs())
    em = (SUM + 36) * U * ad + 2 * U * mean.abs() + U * h.abs().mean(1, keepdim=True)
    er = (40 * U + 2 * U * rms * r) * r
    return (None if residual is None else h, y, torch.cat((mean, r), 1)), (2 * U * h.abs(), ey, torch.cat((em, er), 1))


def layer_norm_backward(h, stats, w, dv, dy):
    """(dh, dw, db) by the formulas from the given stats, and their bounds."""
    N, D = h.shape
    r = stats[:, 1:]
    n = (h - stats[:, :1]) * r
    w = torch.ones(D, dtype=h.dtype) if w is None else w
    t = dy * w
    dh = r * (t - t.mean(1, keepdim=True) - n * (t * n).mean(1, keepdim=True))
    mag = r * (t.abs() + t.abs().mean(1, keepdim=True) + n.abs() * (t * n).abs().mean(1, keepdim=True))
    if dv is not None:
        dh, mag = dh + dv, mag + dv.abs()
    c = N + 80
    return (dh, (dy * n).sum(0), dy.sum(0)), ((SUM + 16) * U * mag, c * U * (dy * n).abs().sum(0), c * U * dy.abs().sum(0))


# ---- linear maps ----
def act(z, name):
    if name == "relu":
        return torch.clamp(z, min=0.0)
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return z * 0.5 * torch.special.erfc(-z / math.sqrt(2.0))
    if name == "gelu_tanh":
        return z * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))
    return z


def slope(z, name):
    """(act'(z), the sum of the magnitudes it is made of), from the formulas."""
    one = torch.ones_like(z)
    if name == "relu":
        return (z > 0).to(z.dtype), one
    if name == "silu":
        s, s1 = torch.sigmoid(z), torch.sigmoid(-z)
        return s + z * s * s1, s + (z * s * s1).abs()
    if name == "gelu":
        q, p = 0.5 * torch.special.erfc(-z / math.sqrt(2.0)), z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
        return q + p, q + p.abs()
    if name == "gelu_tanh":
        a = 2.0 * math.sqrt(2.0 / math.pi)
        u = a * (z + 0.044715 * z ** 3)
        s, s1 = torch.sigmoid(u), torch.sigmoid(-u)
        p = z * a * (1.0 + 3.0 * 0.044715 * z * z) * s * s1
        return s + p, s + p.abs()
    return one, one


def act_rel(z, name, dtype):
    """Relative error of an activation as computed for results of dtype."""
    if name in ("none", "relu"):
        return torch.zeros_like(z)
    if dtype == torch.bfloat16:
        return torch.full_like(z, 2.0 ** -13)
    return (16 + 8 * z * z) * U


def linear(x, w, bias, residual, name, dtype):
    """(y, z) and their bounds: a sum of K products in any order, the activation's own error and its slope (at most
    1.13 in magnitude)."""
    z = x @ w.t()
    ez = (x.shape[1] + 2) * U * (x.abs() @ w.abs().t())
    if bias is not None:
        z, ez = z + bias, ez + 2 * U * bias.abs()
    y = act(z, name)
    ey = 1.13 * ez + act_rel(z, name, dtype) * y.abs()
    if residual is not None:
        y = y + residual
        ey = ey + 2 * U * (y.abs() + residual.abs())
    return (y, z), (ey, ez)


def linear_backward(dy, z, name, dtype):
    """(dz, dbias) and their bounds."""
    s, mag = slope(z, name)
    rel = torch.full_like(z, 2.0 ** -13) if dtype == torch.bfloat16 and name not in ("none", "relu") else (16 + 8 * z * z) * U
    dz = dy * s
    e = dy.abs() * mag * rel
    return (dz, dz.sum(0)), (e, e.sum(0) + (dy.shape[0] + 80) * U * dz.abs().sum(0))


# ---- balance loss and the router's gradient ----
def balance(scores, idx, T, weight, mask):
    """(loss, counts, coef) token by token, and the relative bounds of loss and coef."""
    N, E = scores.shape
    k = idx.shape[1]
    S = (N + T - 1) // T
    counts = torch.zeros((S, E), dtype=torch.int64)
    P = torch.zeros((S, E), dtype=torch.float64)
    V = torch.zeros(S, dtype=torch.float64)
    for n in range(N):
        if mask is not None and not mask[n]:
            continue
        q = n // T
        V[q] += 1
        s = scores[n]
        if s.sum() != 0:
            P[q] += s / s.sum()
        for e in idx[n].tolist():
            if 0 <= e < E:
                counts[q, e] += 1
    V = V.clamp_min(1)[:, None]
    f = E * counts.double() / (k * V)
    coef = weight / S * f / V
    return (weight / S * (f * P / V).sum(), counts, coef), ((T + E + S + 200) * U, 8 * U)


def route_backward(scores, idx, dw, alpha, eps, norm, T=None, coef=None, dloss=1.0, mask=None):
    """dlogits and its bound, token by token."""
    N, E = scores.shape
    out, bound = torch.zeros_like(scores), torch.zeros_like(scores)
    for n in range(N):
        s = scores[n]
        ds, mag = torch.zeros(E, dtype=torch.float64), torch.zeros(E, dtype=torch.float64)
        if dw is not None:
            ok = (idx[n] >= 0) & (idx[n] < E)
            i, g = idx[n][ok].long(), dw[n][ok]
            if norm:
                D = s[i].sum() + eps
                v, m = alpha / D * (g - (g * s[i]).sum() / D), alpha / D * (g.abs() + (g * s[i]).abs().sum() / D)
            else:
                v, m = alpha * g, (alpha * g).abs()
            ds.index_add_(0, i, v)
            mag.index_add_(0, i, m)
        if coef is not None and (mask is None or mask[n]):
            c, t = coef[n // T], s.sum()
            if t != 0:
                ds += dloss * (c - (c * s).sum() / t) / t
                mag += abs(dloss) * (c.abs() + (c * s).abs().sum() / t) / t
        out[n] = ds * s * (1 - s)
        bound[n] = 96 * U * mag * s * (1 - s)
    return out, bound


# ---- gradient norm and clipping ----
def clip(tensors, max_norm, eps):
    """(norm, scale) with the scale from the once-rounded norm."""
    norm = math.sqrt(math.fsum(float(t.double().square().sum()) for t in tensors))
    return norm, min(1.0, max_norm / (norm + eps))


__all__ = ["HALF_STEP", "SUM", "U", "act", "balance", "clip", "layer_norm", "layer_norm_backward", "linear",
           "linear_backward", "route_backward", "slope"]
