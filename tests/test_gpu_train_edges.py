"""Edges of the operators of a training step on the GPU, against float64 references and exact whole-number results."""
import math

import pytest
import torch

import sparse_moe_layer_gate_amd as moe
from tests import _train as R
from tests._ops import check

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
TYPES = {"bf16": BF, "f32": F32}


def gen(seed):
    return torch.Generator().manual_seed(seed)


def workspace(n):
    return torch.empty(max(int(n), 256), dtype=torch.uint8, device="cuda").fill_(0xFF)


# ---------------------------------------------------------------- linear maps
@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("R_,K,M", [(1, 64, 4096), (13, 128, 4096), (40, 704, 328), (300, 64, 520), (65, 4160, 1416),
                                    (2100, 64, 6200), (2100, 192, 6200)])
def test_activation_is_float32_before_the_residual(R_, K, M, act):
    """A residual that takes the activation's bfloat16 value away leaves what float32 knows beyond it: an activation has
    float32's precision wherever it is added to something. Rows of x with a single one make z an element of W, exactly.

    The bound counts steps of U. An exponential's argument is z, z^2 / 2 (gelu) or 1.6 z + 0.07 z^3 (gelu_tanh) and takes five
    rounding steps on its way: below 8 + 8 z^2. The exponential itself, reciprocals, gelu's polynomial of eight terms (the fit,
    what the reciprocal moves it, its own rounding): 24. Then one addition."""
    g = gen(R_ + M)
    x = torch.zeros(R_, K)
    x[torch.arange(R_), torch.arange(R_) * 7 % K] = 1.0
    w = (torch.randn(M, K, generator=g) * 2).clamp(-7, 7).to(BF)
    z = x.double() @ w.double().t()
    a = R.act(z, act)
    res = (-a).to(BF)
    y = torch.empty((R_, M), dtype=BF, device="cuda")
    moe.moe_linear(x.to(BF).cuda(), w.cuda(), y, workspace(moe.moe_linear_workspace_size(R_, K, M)), residual=res.cuda(),
                   act=act)
    ref = a + res.double()
    check("y", y, ref, (32 + 8 * z * z) * R.U * a.abs() + 2 * R.U * ref.abs())


def whole_numbers(g, *shape, most=3, dtype=BF):
    return torch.randint(-most, most + 1, shape, generator=g, device="cuda").to(dtype)


@pytest.mark.parametrize("R_,K,M", [(16400, 64, 32776), (12300, 128, 6152), (6200, 192, 6152), (6200, 256, 6152), (6200, 448, 6152)])
def test_linear_walks_tiles(R_, K, M):
    """More tiles than two rounds of CUs, ragged on both sides, with reductions from one step on: what a block stages for
    one tile is out before the next tile's loads come in. Whole numbers, so every float32 sum is exact."""
    g = torch.Generator(device="cuda").manual_seed(K)
    x, w = whole_numbers(g, R_, K), whole_numbers(g, M, K)
    bias, res = whole_numbers(g, M, most=50), whole_numbers(g, R_, M, most=50)
    sums = x.float() @ w.float().t() + bias.float()
    ws = workspace(moe.moe_linear_workspace_size(R_, K, M))
    for parts in ("", "z", "br", "brz"):
        y = torch.full((R_, M), float("nan"), dtype=BF, device="cuda")
        z = torch.full((R_, M), float("nan"), dtype=BF, device="cuda") if "z" in parts else None
        moe.moe_linear(x, w, y, ws, bias=bias if "b" in parts else None, residual=res if "r" in parts else None, act="relu",
                       z=z)
        zz = sums if "b" in parts else sums - bias.float()
        assert z is None or torch.equal(z, zz.to(BF))
        ref = torch.relu(zz)
        assert torch.equal(y, (ref + res.float() if "r" in parts else ref).to(BF))


def test_linear_outputs_before_and_behind_4_gib():
    """4.6 GB of y, every row compared, from an output that held no numbers."""
    g = torch.Generator(device="cuda").manual_seed(90)
    R_, K, M = 70000, 192, 32776
    x, w = whole_numbers(g, R_, K), whole_numbers(g, M, K)
    y = torch.full((R_, M), float("nan"), dtype=BF, device="cuda")
    moe.moe_linear(x, w, y, workspace(moe.moe_linear_workspace_size(R_, K, M)), act="relu")
    for at in range(0, R_, 8192):
        assert torch.equal(y[at:at + 8192], torch.relu(x[at:at + 8192].float() @ w.float().t()).to(BF))


# ---------------------------------------------------------------- gradient norm and clipping
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_clip_of_zeros_to_nothing(dtype):
    """No ratio below 1 leaves the scale 1, 0 / 0 too: zeros stay zeros. A NaN in the norm still shows."""
    dt = TYPES[dtype]
    ts = [torch.zeros(n, dtype=dt, device="cuda") for n in (5, 3000, 5000000)]
    norm = torch.full((1,), float("nan"), device="cuda")
    moe.moe_grad_norm(ts, norm, workspace(moe.moe_grad_norm_workspace_size(ts)))
    assert float(norm) == 0
    out = [torch.full_like(t, 7.0) for t in ts]
    moe.moe_grad_clip(ts, norm, 0.0, out=out, eps=0.0)
    moe.moe_grad_clip(ts, norm, 0.0, eps=0.0)
    for t, o in zip(ts, out):
        assert (t == 0).all() and (o == 0).all()
    ts[0].fill_(3.0)  # a norm above 0: nothing is left
    norm.fill_(3.0 * math.sqrt(5))
    moe.moe_grad_clip(ts, norm, 0.0, eps=0.0)
    assert (ts[0] == 0).all()
    norm.fill_(float("nan"))
    moe.moe_grad_clip(ts, norm, 0.0, eps=0.0)
    assert ts[1].isnan().all()


def test_norm_does_not_depend_on_the_place():
    """The same values at any address give the same bits. The sum of these squares lies on the border between two float32
    norms: two of them, each less than half a step of the sum, add to it only where they meet before the large one."""
    x = torch.zeros(1900)
    x[0], x[800], x[1600], x[1200], x[400] = 1.0, 2.0 ** -12, 2.0 ** -12, 2.0 ** -24, 2.0 ** -26
    x[1] = x[2] = math.sqrt(0.98 * 2.0 ** -53)
    for dt in (F32, BF):
        v = x.to(dt).cuda()
        norms = []
        for at in range(70):
            buf = torch.full((x.numel() + 128,), 5.0, dtype=dt, device="cuda")
            t = buf[at:at + x.numel()]
            t.copy_(v)
            norm = torch.empty(1, device="cuda")
            moe.moe_grad_norm([t], norm, workspace(moe.moe_grad_norm_workspace_size([t])))
            norms.append(float(norm))
        assert len(set(norms)) == 1, norms


def clip_sizes(chunk, at, line):
    """Lengths of tensors that lie end to end from value `at` on, so that with what precedes each in its line of `line`
    values they fill whole chunks, miss one by a value or exceed it by one; more than a launch's table holds."""
    sizes = []
    for i in range(130):
        lead = at % line
        n = [chunk - 1 - lead, chunk - lead, chunk + 1 - lead, 3 * chunk - lead, 1, 2 * chunk - 1 - lead, 7, 4 * chunk + 1 - lead,
             0, 2 * chunk + 77][i % 10]
        sizes.append(n)
        at += n
    return sizes


@pytest.mark.parametrize("flat", [False, True])
@pytest.mark.parametrize("dtype,to", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("chunk", [2048, 8192])
def test_clip_around_chunks(chunk, dtype, to, flat):
    """Both chunk lengths (lists of up to 4 M values and longer ones) at their edges, every value and what lies around."""
    dt, ot = TYPES[dtype], TYPES[to]
    line = 128 // (2 if ot == BF else 4)
    g = torch.Generator(device="cuda").manual_seed(chunk)
    sizes = clip_sizes(chunk, 5, line if flat else 1)
    if chunk == 8192:
        sizes[60] += 3000000
        assert sum(sizes) > 1 << 22
    else:
        assert sum(sizes) < 1 << 22
    total = sum(sizes)
    print(f"[clip] {len(sizes)} tensors, {total} values {dtype} -> {to} flat={flat}", flush=True)
    if flat:
        whole = torch.randn(total + 100, generator=g, device="cuda").mul_(0.1).to(dt)
        grads = list(whole[5:5 + total].split(sizes))
        buf = torch.full((total + 100,), 7.0, dtype=ot, device="cuda")
        out = list(buf[5:5 + total].split(sizes))
    else:
        grads = [torch.randn(n, generator=g, device="cuda").mul_(0.1).to(dt) for n in sizes]
        out = [torch.full((n,), 7.0, dtype=ot, device="cuda") for n in sizes]
    before = [t.clone() for t in grads]
    norm = torch.full((1,), float("nan"), device="cuda")
    moe.moe_grad_norm(grads, norm, workspace(moe.moe_grad_norm_workspace_size(grads)))
    rn, scale = R.clip([t.cpu() for t in before], 0.25, 1e-6)
    assert abs(float(norm) - rn) <= 1.0001 * R.U * rn
    moe.moe_grad_clip(grads, norm, 0.25, out=out)
    flat_in, flat_out = torch.cat(before).cpu().double(), torch.cat(out)
    check("out", flat_out, flat_in * scale, 4 * R.U * (flat_in * scale).abs())
    for a, b in zip(grads, before):
        assert torch.equal(a, b)
    if flat:
        assert (buf[:5] == 7).all() and (buf[5 + total:] == 7).all()
    if dt == ot:
        edge = [whole[:5].clone(), whole[5 + total:].clone()] if flat else []
        moe.moe_grad_clip(grads, norm, 0.25)
        assert torch.equal(torch.cat(grads), flat_out)
        if flat:
            assert torch.equal(whole[:5], edge[0]) and torch.equal(whole[5 + total:], edge[1])


# ---------------------------------------------------------------- balance loss and the router's gradient
@pytest.mark.parametrize("eps", [1e-20, 0.0])
@pytest.mark.parametrize("N,E,k,T", [(12, 6, 2, 5), (40, 32, 4, 40), (40, 160, 8, 10), (40, 130, 8, 13), (1100, 512, 8, 700),
                                     (9, 257, 1, 9)])
def test_scores_whose_sum_has_no_float32_reciprocal(N, E, k, T, eps):
    """Tokens whose scores are subnormal have the shares of any other token, down to one expert's least score above 0."""
    g = gen(N + E)
    scores = torch.rand((N, E), generator=g) * 0.9 + 0.05
    scores[1::4] *= 1e-40 / E
    scores[2] = 2.0 ** -149
    scores[3] = 0.0
    scores[3, E // 2] = 2.0 ** -149
    scores[4::16] = 0.0
    scores[5, :] = 2.0 ** -149
    scores[5, 0] = 0.75
    idx = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(N)]).to(torch.int32)
    idx[3, 0] = E // 2
    idx[3, 1:] = -1
    dw = torch.randn((N, k), generator=g)
    cfg, S = moe.make_config(64, E, 1, 1, k, 64, eps=eps), (N + T - 1) // T
    s, i = scores.cuda(), idx.cuda()
    counts, coef, loss = (torch.empty((S, E), dtype=torch.int32, device="cuda"), torch.empty((S, E), device="cuda"),
                          torch.empty(1, device="cuda"))
    moe.moe_balance_loss(cfg, N, s, i, T, 0.5, counts, coef, loss, workspace(moe.moe_balance_workspace_size(cfg, N, T)))
    (rl, rc, rf), (el, ef) = R.balance(scores.double(), idx, T, 0.5, None)
    assert torch.equal(counts.cpu().long(), rc)
    check("loss", loss, rl.view(1), el * rl.abs().view(1))
    check("coef", coef, rf, ef * rf.abs())
    c = coef.cpu().double()
    for norm in (True, False):
        cfg = moe.make_config(64, E, 1, 1, k, 64, eps=eps, norm=norm)
        e = float(torch.tensor(eps))  # as float32 holds it
        for wts, co in ((None, c), (dw, None), (dw, c)):
            if norm and eps == 0 and wts is not None:
                wts = wts.clone()
                wts[4::16] = 0.0  # 0 / 0 in the formula
            out = torch.empty((N, E), device="cuda")
            moe.moe_route_backward(cfg, N, s, i, None if wts is None else wts.cuda(), out, seq_rows=T,
                                   coef=None if co is None else coef)
            ref, bound = R.route_backward(scores.double(), idx, None if wts is None else wts.double(), 1.0, e, norm, T, co)
            dead = ~ref.isfinite()  # the formula's 0 / 0: weights of scores that sum to 0, without eps
            assert not dead.any() or (norm and eps == 0 and wts is not None)
            assert (out.cpu()[dead] == 0).all()
            ref[dead], bound[dead] = 0.0, 0.0
            check("dlogits", out, ref, bound)
