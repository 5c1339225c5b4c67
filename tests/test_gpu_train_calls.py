"""The operators of a training step as a program uses them: one after the other in a training step, captured into a graph and
replayed, on other streams, at the same time, twice with the same bits, and on tensors of more than 4 GiB."""
import pytest
import torch

import sparse_moe_layer_gate_amd as moe
from tests import _ops as O
from tests import _train as R

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
TYPES = {"bf16": BF, "f32": F32}


def gen(seed):
    return torch.Generator().manual_seed(seed)


def workspace(n):
    return torch.empty(max(int(n), 256), dtype=torch.uint8, device="cuda").fill_(0xFF)


def empty(*shape, dtype=F32):
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


# ---------------------------------------------------------------- a training step
def test_training_step():
    """Residual and layer norm, two linear maps, router with its balance loss, routed experts, their combine: the gradients of
    every weight and of the input, and their clipping, against autograd of the same step in float64.

    Float32. Each of the ten operators on a gradient's way adds at most (sum length + 100) U of the magnitudes it adds up,
    here below 400 U = 2.4e-5; with magnitudes up to ten times the result's norm and ten operators, 2.4e-3."""
    N, D, Fd, E, k, T = 96, 128, 256, 8, 2, 32
    g = gen(71)

    def rand(*s, std=1.0):
        return torch.randn(s, generator=g) * std
    p = {"x": rand(N, D), "r": rand(N, D), "lw": 1 + 0.1 * rand(D), "lb": 0.1 * rand(D),
         "w1": rand(Fd, D, std=D ** -0.5), "b1": 0.1 * rand(Fd), "w2": rand(D, Fd, std=Fd ** -0.5), "b2": 0.1 * rand(D),
         "wg": rand(E, D, std=D ** -0.5), "we": rand(E, D, D, std=D ** -0.5)}
    gy = rand(N, D)
    weight, dloss = 0.5, 2.0
    cfg = moe.make_config(D, E, 1, 1, k, 64, alpha=1.5, dtype="f32")
    d = {n: v.cuda() for n, v in p.items()}
    one = torch.tensor([0, N], dtype=torch.int32, device="cuda")
    ws = workspace(max(moe.moe_linear_workspace_size(N, D, Fd, "f32"), moe.moe_linear_workspace_size(N, Fd, D, "f32"),
                       moe.moe_linear_backward_workspace_size(N, Fd, "f32"), moe.moe_layer_norm_workspace_size(N, D, "f32"),
                       moe.moe_grouped_workspace_size(E, N * k, "f32"), moe.moe_grouped_workspace_size(1, N, "f32"),
                       moe.moe_balance_workspace_size(cfg, N, T), moe.moe_workspace_size(cfg, N),
                       moe.moe_dispatch_workspace_size(cfg, N)))
    # forward
    h, u, stats, z1, a1, o = empty(N, D), empty(N, D), empty(N, 2), empty(N, Fd), empty(N, Fd), empty(N, D)
    moe.moe_layer_norm(N, d["x"], d["r"], d["lw"], d["lb"], h, u, stats)
    moe.moe_linear(u, d["w1"], a1, ws, bias=d["b1"], act="gelu", z=z1)
    moe.moe_linear(a1, d["w2"], o, ws, bias=d["b2"], residual=h)
    scores, tw = empty(N, E), empty(N, k)
    ti = torch.empty((N, k), dtype=torch.int32, device="cuda")
    moe.moe_route(cfg, N, o, d["wg"], torch.zeros(E, device="cuda"), scores, ti, tw, flags=moe.MOE_ROUTE_SCORES_OUT,
                  workspace=ws)
    counts, offsets = (torch.empty(n, dtype=torch.int32, device="cuda") for n in (E, E + 1))
    pair, inv = (torch.empty(N * k, dtype=torch.int32, device="cuda") for _ in range(2))
    moe.moe_dispatch(cfg, N, ti, counts, offsets, pair, inv, ws)
    S = N // T
    seq_counts, coef, loss = torch.empty((S, E), dtype=torch.int32, device="cuda"), empty(S, E), empty(1)
    moe.moe_balance_loss(cfg, N, scores, ti, T, weight, seq_counts, coef, loss, ws)
    rows, y = empty(N * k, D), empty(N, D)
    moe.moe_grouped_linear(o, d["we"], offsets, rows, ws, row_index=pair, index_div=k)
    moe.moe_combine(N, k, rows, inv, tw, o, y)
    assert torch.equal(seq_counts.sum(0), counts)
    # backward
    gr = {n: empty(*v.shape) for n, v in d.items()}
    dy = gy.cuda()
    drows, dtw, dxr, dlog = empty(N * k, D), empty(N, k), empty(N * k, D), empty(N, E)
    moe.moe_combine_backward(N, k, dy, rows, inv, tw, drows, dtw)
    moe.moe_grouped_linear_wgrad(drows, o, offsets, gr["we"], ws, row_index=pair, index_div=k)
    moe.moe_grouped_linear_dgrad(drows, d["we"], offsets, dxr, ws)
    moe.moe_route_backward(cfg, N, scores, ti, dtw, dlog, seq_rows=T, coef=coef,
                           dloss=torch.full((1,), dloss, device="cuda"))
    gr["wg"] = dlog.t().mm(o)
    do = empty(N, D)
    moe.moe_combine(N, k, dxr, inv, None, dy + dlog.mm(d["wg"]), do)
    moe.moe_linear_backward(do, None, None, gr["b2"], ws)
    da, dz1, du, dx = empty(N, Fd), empty(N, Fd), empty(N, D), empty(N, D)
    moe.moe_grouped_linear_wgrad(do, a1, one, gr["w2"].view(1, D, Fd), ws)
    moe.moe_grouped_linear_dgrad(do, d["w2"].view(1, D, Fd), one, da, ws)
    moe.moe_linear_backward(da, z1, dz1, gr["b1"], ws, act="gelu")
    moe.moe_grouped_linear_wgrad(dz1, u, one, gr["w1"].view(1, Fd, D), ws)
    moe.moe_grouped_linear_dgrad(dz1, d["w1"].view(1, Fd, D), one, du, ws)
    moe.moe_layer_norm_backward(N, h, stats, d["lw"], do, du, dx, gr["lw"], gr["lb"], ws)
    gr["x"] = gr["r"] = dx
    # the same step in float64, the routing as chosen
    q = {n: v.double().requires_grad_() for n, v in p.items()}
    hh = q["x"] + q["r"]
    m = hh - hh.mean(1, keepdim=True)
    uu = m / torch.sqrt(m.square().mean(1, keepdim=True) + 1e-5) * q["lw"] + q["lb"]
    oo = R.act(uu @ q["w1"].t() + q["b1"], "gelu") @ q["w2"].t() + q["b2"] + hh
    s = torch.sigmoid(oo @ q["wg"].t())
    idx = ti.cpu().long()
    chosen = s.gather(1, idx)
    wt = 1.5 * chosen / (chosen.sum(1, keepdim=True) + 1e-20)
    ex = torch.stack([torch.stack([q["we"][int(e)] @ oo[n] for e in idx[n]]) for n in range(N)])
    yy = (wt[..., None] * ex).sum(1) + oo
    prob = s / s.sum(1, keepdim=True)
    f = torch.stack([torch.bincount(idx[i:i + T].reshape(-1), minlength=E) for i in range(0, N, T)]).double() * E / (k * T)
    ll = weight / S * (f * prob.view(S, T, E).mean(1)).sum()
    ((yy * gy.double()).sum() + dloss * ll).backward()

    def near(name, got, ref):
        err = float((got.cpu().double() - ref).norm() / ref.norm())
        print(f"  {name}: {err:.3g}", flush=True)
        assert err < 2.4e-3, name
    near("y", y, yy.detach())
    near("loss", loss, ll.detach().view(1))
    for n in p:
        near("d" + n, gr[n], q[n].grad)
    # clipping of all weights' gradients
    names = [n for n in p if n not in ("x", "r")]
    lst = moe.moe_tensor_list([gr[n] for n in names])
    norm = empty(1)
    before = [gr[n].clone() for n in names]
    moe.moe_grad_norm(lst, norm, workspace(moe.moe_grad_norm_workspace_size(lst)))
    moe.moe_grad_clip(lst, norm, 1.0)
    rn, scale = R.clip([t.cpu() for t in before], 1.0, 1e-6)
    assert abs(float(norm) - rn) <= 1.0001 * R.U * rn and scale < 1
    for n, b in zip(names, before):
        O.check(n, gr[n], b.cpu().double() * scale, 4 * R.U * b.cpu().double().abs())


# ---------------------------------------------------------------- calls of every operator
class Calls:
    """One call of each operator and direction on buffers of its own; `run` enqueues them all."""

    def __init__(self, seed, dtype="bf16", N=300, D=320, M=520, E=48, k=4):
        dt, g = TYPES[dtype], gen(seed)

        def rand(*s, t=dt):
            return torch.randn(s, generator=g).to(t).cuda()
        self.N, self.k, self.T = N, k, 70
        self.x, self.r, self.w, self.b, self.dy, self.dv = rand(N, D), rand(N, D), rand(D), rand(D), rand(N, D), rand(N, D)
        self.wm, self.bm, self.res, self.dm = rand(M, D), rand(M), rand(N, M), rand(N, M)
        self.few, self.long = rand(5, D), rand(N, 2048)
        self.wlong = rand(M, 2048)
        self.scores = torch.sigmoid(rand(N, E, t=F32))
        self.idx = self.scores.topk(k, 1).indices.to(torch.int32)
        self.dw = rand(N, k, t=F32)
        self.mask = (torch.rand(N, generator=g) < 0.8).cuda()
        self.cfg = moe.make_config(64, E, 1, 1, k, 64)
        S = (N + self.T - 1) // self.T
        self.out = {"h": empty(N, D, dtype=dt), "u": empty(N, D, dtype=dt), "stats": empty(N, 2), "dh": empty(N, D, dtype=dt),
                    "lw": empty(D), "lb": empty(D), "y": empty(N, M, dtype=dt), "z": empty(N, M, dtype=dt),
                    "yf": empty(5, M, dtype=dt), "yl": empty(N, M, dtype=dt), "dz": empty(N, M, dtype=dt), "db": empty(M),
                    "loss": empty(1), "coef": empty(S, E), "dlog": empty(N, E), "norm": empty(1),
                    "counts": torch.full((S, E), -1, dtype=torch.int32, device="cuda"),
                    "c0": empty(N, D), "c1": empty(M)}
        self.grads = moe.moe_tensor_list([self.dy, self.bm])
        self.clipped = moe.moe_tensor_list([self.out["c0"], self.out["c1"]])
        sizes = [moe.moe_layer_norm_workspace_size(N, D, dtype), moe.moe_linear_workspace_size(N, D, M, dtype),
                 moe.moe_linear_workspace_size(N, 2048, M, dtype), moe.moe_linear_backward_workspace_size(N, M, dtype),
                 moe.moe_balance_workspace_size(self.cfg, N, self.T), moe.moe_grad_norm_workspace_size(self.grads)]
        self.ws = workspace(max(sizes))  # one for all: the calls run one after the other

    def run(self, stream=None):
        o, s = self.out, dict(stream=stream)
        moe.moe_layer_norm(self.N, self.x, self.r, self.w, self.b, o["h"], o["u"], o["stats"], **s)
        moe.moe_layer_norm_backward(self.N, o["h"], o["stats"], self.w, self.dv, self.dy, o["dh"], o["lw"], o["lb"], self.ws, **s)
        moe.moe_linear(o["u"], self.wm, o["y"], self.ws, bias=self.bm, residual=self.res, act="gelu_tanh", z=o["z"], **s)
        moe.moe_linear(self.few, self.wm, o["yf"], None, bias=self.bm, act="silu", **s)
        moe.moe_linear(self.long, self.wlong, o["yl"], self.ws, act="relu", **s)
        moe.moe_linear_backward(self.dm, o["z"], o["dz"], o["db"], self.ws, act="gelu", **s)
        moe.moe_balance_loss(self.cfg, self.N, self.scores, self.idx, self.T, 0.1, o["counts"], o["coef"], o["loss"], self.ws,
                             token_mask=self.mask, **s)
        moe.moe_route_backward(self.cfg, self.N, self.scores, self.idx, self.dw, o["dlog"], seq_rows=self.T, coef=o["coef"],
                               dloss=o["loss"], token_mask=self.mask, **s)
        moe.moe_grad_norm(self.grads, o["norm"], self.ws, **s)
        moe.moe_grad_clip(self.grads, o["norm"], 3.0, out=self.clipped, **s)

    def results(self):
        torch.cuda.synchronize()
        return {n: t.clone() for n, t in self.out.items()}

    def spoil(self):
        for t in self.out.values():
            t.fill_(7)
        self.ws.fill_(0xFF)


def same(a, b):
    for n in a:
        assert torch.equal(a[n], b[n]), n


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_same_bits_again(dtype):
    c = Calls(81, dtype)
    c.run()
    first = c.results()
    for t in first.values():
        assert t.double().isfinite().all()
    c.spoil()
    c.run()
    same(first, c.results())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_captured_and_replayed(dtype):
    """Every call in one graph: replays with other inputs in the same buffers, eager work of the same operators in between,
    all with the bits of the eager calls."""
    c, other = Calls(82, dtype), Calls(83, dtype)
    c.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run()
    for turn in range(4):
        for t in (c.x, c.r, c.dy, c.dm, c.long, c.few):
            t.copy_(torch.randn(t.shape, generator=gen(90 + turn)).to(t.dtype))
        c.spoil()
        graph.replay()
        got = c.results()
        other.run()
        torch.cuda.synchronize()
        c.spoil()
        c.run()
        same(got, c.results())


def test_other_stream_given_and_current():
    c = Calls(84)
    c.run()
    ref = c.results()
    side = torch.cuda.Stream()
    c.spoil()
    torch.cuda.synchronize()
    c.run(stream=side)  # given: not the current one
    side.synchronize()
    same(ref, c.results())
    c.spoil()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        c.run()
    side.synchronize()
    same(ref, c.results())


def test_two_streams_at_once():
    a, b = Calls(85), Calls(86, "f32")
    a.run()
    b.run()
    ra, rb = a.results(), b.results()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    a.spoil()
    b.spoil()
    torch.cuda.synchronize()
    for _ in range(5):
        a.run(stream=sa)
        b.run(stream=sb)
    same(ra, a.results())
    same(rb, b.results())


# ---------------------------------------------------------------- more than 4 GiB
def test_rows_behind_4_gib():
    """The last rows of tensors of more than 2^32 bytes and 2^31 values, against a call on those rows alone."""
    D, n = 8192, 64
    N = (1 << 18) + 4096 + n  # 2.2e9 values, 4.4 GB
    g = torch.Generator(device="cuda").manual_seed(87)
    x = torch.empty((N, D), dtype=BF, device="cuda")
    for i in range(0, N, 1 << 15):
        x[i:i + (1 << 15)].normal_(generator=g)
    w, b = (torch.randn(D, generator=g, device="cuda").to(BF) for _ in range(2))
    y, stats = torch.empty_like(x), torch.empty((N, 2), device="cuda")
    moe.moe_layer_norm(N, x, None, w, b, None, y, stats)
    ys, ss = torch.empty((n, D), dtype=BF, device="cuda"), torch.empty((n, 2), device="cuda")
    moe.moe_layer_norm(n, x[-n:], None, w, b, None, ys, ss)
    assert torch.equal(y[-n:], ys) and torch.equal(stats[-n:], ss)
    moe.moe_layer_norm_backward(N, x, stats, w, None, y, y2 := torch.empty_like(x), None, None, None)
    moe.moe_layer_norm_backward(n, x[-n:], ss, w, None, ys, ys2 := torch.empty_like(ys), None, None, None)
    assert torch.equal(y2[-n:], ys2)
    # the epilogue's gradients and the clip over the same memory
    ws = workspace(moe.moe_linear_backward_workspace_size(N, D))
    db = torch.empty(D, device="cuda")
    moe.moe_linear_backward(x, y, y2, db, ws, act="silu")
    moe.moe_linear_backward(x[-n:], y[-n:], ys2, None, None, act="silu")
    assert torch.equal(y2[-n:], ys2) and db.isfinite().all()
    norm = torch.empty(1, device="cuda")
    moe.moe_grad_norm([x], norm, workspace(moe.moe_grad_norm_workspace_size([x])))
    assert abs(float(norm) / (N * D) ** 0.5 - 1) < 1e-3  # of unit normal values: 1 to within a few 1 / sqrt(2 N D)
    tail = x[-n:].clone()
    moe.moe_grad_clip([x], norm, 0.5 * float(norm), eps=0.0)
    assert torch.equal(x[-n:], tail * 0.5)


def test_linear_outputs_behind_4_gib():
    """4.6 GB of y from 256 x 256 tiles, and 8.6 GB of W under few rows and under small tiles."""
    g = torch.Generator(device="cuda").manual_seed(88)
    Rr, K, M, n = 70000, 64, 32776, 100
    x = torch.randint(-3, 4, (Rr, K), generator=g, device="cuda").to(BF)
    w = torch.randint(-3, 4, (M, K), generator=g, device="cuda").to(BF)
    y = torch.empty((Rr, M), dtype=BF, device="cuda")
    ws = workspace(max(moe.moe_linear_workspace_size(Rr, K, M), 1 << 25))
    moe.moe_linear(x, w, y, ws, act="relu")
    ref = torch.relu(x[-n:].float() @ w.float().t()).to(BF)  # whole numbers: exact
    assert torch.equal(y[-n:], ref)
    del y
    K, M = 2048, (1 << 20) - 8
    w = torch.empty((M, K), dtype=F32, device="cuda")
    for i in range(0, M, 1 << 16):
        w[i:i + (1 << 16)] = torch.randint(-3, 4, w[i:i + (1 << 16)].shape, generator=g, device="cuda").float()
    for rows in (3, 40):
        x = torch.randint(-3, 4, (rows, K), generator=g, device="cuda").float()
        y = torch.empty((rows, M), device="cuda")
        moe.moe_linear(x, w, y, ws)
        assert torch.equal(y[:, -2000:], x @ w[-2000:].t())


def test_balance_rows_behind_4_gib():
    N, E, k, n = (1 << 22) + 700, 512, 2, 512
    g = torch.Generator(device="cuda").manual_seed(89)
    scores = torch.rand((N, E), generator=g, device="cuda")
    idx = torch.randint(0, E, (N, k), generator=g, device="cuda", dtype=torch.int32)
    cfg = moe.make_config(64, E, 1, 1, k, 64)
    dw = torch.randn((N, k), generator=g, device="cuda")
    T = 1 << 16
    S = (N + T - 1) // T
    counts, coef, loss = torch.empty((S, E), dtype=torch.int32, device="cuda"), empty(S, E), empty(1)
    moe.moe_balance_loss(cfg, N, scores, idx, T, 1.0, counts, coef, loss, workspace(moe.moe_balance_workspace_size(cfg, N, T)))
    assert torch.equal(counts.sum(0).long(), torch.bincount(idx.view(-1), minlength=E))
    assert torch.equal(counts[-1].long(), torch.bincount(idx[(S - 1) * T:].reshape(-1), minlength=E))
    out = torch.empty_like(scores)
    moe.moe_route_backward(cfg, N, scores, idx, dw, out, seq_rows=T, coef=coef)
    last = empty(n, E)
    moe.moe_route_backward(cfg, n, scores[-n:], idx[-n:], dw[-n:], last, seq_rows=n, coef=coef[-1:])
    assert torch.equal(out[-n:], last)


# ---------------------------------------------------------------- nothing outside
class Guarded:
    """Outputs and workspaces between runs of a known byte, which no call may change."""

    def __init__(self):
        self.all = []

    def __call__(self, shape, dtype=F32):
        n = torch.empty(shape, dtype=dtype).nbytes
        buf = torch.full((n + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
        self.all.append((buf, n))
        return buf[4096:4096 + n].view(dtype).view(shape)

    def workspace(self, n):
        return self((n,), torch.uint8) if n else None

    def check(self):
        torch.cuda.synchronize()
        for buf, n in self.all:
            assert (buf[:4096] == 0xA5).all() and (buf[4096 + n:] == 0xA5).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,D", [(1, 8), (5, 264), (67, 1032), (301, 2568), (33, 5128), (9, 12296)])
def test_layer_norm_writes_its_outputs_alone(N, D, dtype):
    dt, g, out = TYPES[dtype], gen(N + D), Guarded()
    x, r, dy = (torch.randn(N, D, generator=g).to(dt).cuda() for _ in range(3))
    w = torch.randn(D, generator=g).to(dt).cuda()
    h, y, dh, stats, dw, db = out((N, D), dt), out((N, D), dt), out((N, D), dt), out((N, 2)), out((D,)), out((D,))
    moe.moe_layer_norm(N, x, r, w, w, h, y, stats)
    moe.moe_layer_norm_backward(N, h, stats, w, r, dy, dh, dw, db,
                                out.workspace(moe.moe_layer_norm_workspace_size(N, D, dtype)))
    out.check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("R_,K,M", [(1, 64, 8), (13, 704, 40), (45, 512, 136), (66, 1024, 264), (66, 64, 8304), (145, 256, 11000),
                                    (133, 3456, 5528), (140, 896, 11120), (2100, 256, 6200), (3722, 7232, 272)])
def test_linear_writes_its_outputs_alone(R_, K, M, dtype):
    dt, g, out = TYPES[dtype], gen(R_ + M), Guarded()
    x, w = torch.randn(R_, K, generator=g).to(dt).cuda(), torch.randn(M, K, generator=g).to(dt).cuda()
    y, z, dz, db = out((R_, M), dt), out((R_, M), dt), out((R_, M), dt), out((M,))
    moe.moe_linear(x, w, y, out.workspace(moe.moe_linear_workspace_size(R_, K, M, dtype)), act="silu", z=z)
    moe.moe_linear_backward(y, z, dz, db, out.workspace(moe.moe_linear_backward_workspace_size(R_, M, dtype)), act="silu")
    out.check()


@pytest.mark.parametrize("N,E,k,T", [(1, 1, 1, 1), (77, 6, 2, 20), (100, 60, 8, 100), (1500, 130, 4, 1400), (4000, 256, 8, 1000),
                                     (9000, 32, 32, 9000), (70000, 64, 6, 1024), (600, 512, 8, 2)])
def test_balance_writes_its_outputs_alone(N, E, k, T):
    g, out = gen(N + E), Guarded()
    scores = torch.rand(N, E, generator=g).cuda()
    idx = torch.randint(-1, E + 1, (N, k), generator=g, dtype=torch.int32).cuda()
    cfg, S = moe.make_config(64, E, 1, 1, k, 64), (N + T - 1) // T
    counts, coef, loss, d = out((S, E), torch.int32), out((S, E)), out((1,)), out((N, E))
    moe.moe_balance_loss(cfg, N, scores, idx, T, 0.1, counts, coef, loss,
                         out.workspace(moe.moe_balance_workspace_size(cfg, N, T)))
    moe.moe_route_backward(cfg, N, scores, idx, torch.randn(N, k, generator=g).cuda(), d, seq_rows=T, coef=coef)
    out.check()


def test_norm_workspace_of_its_size():
    out = Guarded()
    for sizes in ([1], [2048] * 3, [5, 70000, 1], [5000000, 9]):
        grads = [torch.ones(n + 1, device="cuda")[1:] for n in sizes]
        norm = out((1,))
        moe.moe_grad_norm(grads, norm, out.workspace(moe.moe_grad_norm_workspace_size(grads)))
        assert abs(float(norm) / sum(sizes) ** 0.5 - 1) < 1e-6
    out.check()


def test_no_rows():
    """Calls without rows write the sums over none and nothing else."""
    out = Guarded()
    cfg = moe.make_config(64, 16, 1, 1, 2, 64)
    none, dw, db, dbias, loss = out((0, 64)), out((64,)), out((64,)), out((64,)), out((1,))
    moe.moe_layer_norm(0, none, None, None, None, None, none)
    moe.moe_layer_norm_backward(0, none, out((0, 2)), None, None, none, none, dw, db, None)
    moe.moe_linear(none, torch.ones(64, 64, device="cuda"), none)
    moe.moe_linear_backward(none, none, none, dbias, None, act="gelu")
    moe.moe_linear_backward(none, none, none, None, None, act="gelu")
    moe.moe_balance_loss(cfg, 0, out((0, 16)), out((0, 2), torch.int32), 4, 1.0, None, None, loss, None)
    moe.moe_route_backward(cfg, 0, out((0, 16)), out((0, 2), torch.int32), out((0, 2)), out((0, 16)))
    out.check()
    for t in (dw, db, dbias, loss):
        assert (t == 0).all()
