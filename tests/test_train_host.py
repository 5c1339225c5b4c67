"""The operators of a training step without a GPU: argument errors are found on the host before any launch, sizes
never fall, and the Python binding refuses what is not a device tensor of the right type and shape."""
import ctypes

import numpy as np
import pytest
import torch

import sparse_moe_layer_gate_amd as moe

INV, UNS, WS, OK = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED, moe.MOE_ERR_WORKSPACE, moe.MOE_OK
BIG = 1 << 60
I63 = (1 << 63) - 1
NAN, INF = float("nan"), float("inf")


def p(i):
    return ctypes.c_void_p(4096 * (i + 1))  # never dereferenced


ODD = ctypes.c_void_p(4100)


def ln(N=4, D=256, dt=moe.MOE_BF16, eps=1e-5, x=p(0), res=p(1), w=p(2), b=p(3), h=p(4), y=p(5), st=p(6)):
    return moe.lib().moe_layer_norm(N, D, dt, eps, x, res, w, b, h, y, st, None)


def ln_bwd(N=4, D=256, dt=moe.MOE_BF16, h=p(0), st=p(1), w=p(2), dv=p(3), dy=p(4), dh=p(5), dw=p(6), db=p(7), ws=p(8), n=BIG):
    return moe.lib().moe_layer_norm_backward(N, D, dt, h, st, w, dv, dy, dh, dw, db, ws, n, None)


@pytest.mark.parametrize("fn,kw,status", [
    (ln, dict(N=-1), INV), (ln, dict(D=0), INV), (ln, dict(D=12), UNS), (ln, dict(D=16392), UNS), (ln, dict(N=1 << 31), UNS),
    (ln, dict(N=I63), UNS), (ln, dict(dt=2), INV), (ln, dict(eps=-1.0), INV), (ln, dict(eps=NAN), INV), (ln, dict(x=None), INV),
    (ln, dict(y=None), INV), (ln, dict(h=None), INV), (ln, dict(res=None), INV), (ln, dict(y=p(0)), INV),
    (ln, dict(y=p(1)), INV), (ln, dict(y=p(4)), INV), (ln, dict(x=ODD), INV), (ln, dict(st=ODD), INV),
    (ln, dict(N=0, x=None), OK),
    # a row's threads: 8, 64, 512
    (ln, dict(N=1 << 29, D=64), UNS), (ln, dict(N=1 << 26, D=512), UNS), (ln, dict(N=1 << 23, D=16384), UNS),
    (ln_bwd, dict(N=-1), INV), (ln_bwd, dict(D=20), UNS), (ln_bwd, dict(h=None), INV), (ln_bwd, dict(st=None), INV),
    (ln_bwd, dict(dy=None), INV), (ln_bwd, dict(dh=None), INV), (ln_bwd, dict(dh=p(0)), INV), (ln_bwd, dict(dh=p(4)), INV),
    (ln_bwd, dict(db=p(6)), INV), (ln_bwd, dict(dw=ODD), INV), (ln_bwd, dict(ws=None), WS), (ln_bwd, dict(n=4095), WS),
    (ln_bwd, dict(ws=ctypes.c_void_p(8)), WS), (ln_bwd, dict(db=None, ws=None), WS), (ln_bwd, dict(N=1 << 31), UNS),
    (ln_bwd, dict(N=0, dw=None, db=None), OK),
])
def test_layer_norm_errors(fn, kw, status):
    assert fn(**kw) == status


def lin(R=4, K=256, M=128, dt=moe.MOE_BF16, act=1, x=p(0), w=p(1), b=p(2), res=p(3), z=p(4), y=p(5), ws=p(6), n=BIG):
    return moe.lib().moe_linear(R, K, M, dt, act, x, w, b, res, z, y, ws, n, None)


def lin_bwd(R=4, M=128, dt=moe.MOE_BF16, act=1, dy=p(0), z=p(1), dz=p(2), db=p(3), ws=p(4), n=BIG):
    return moe.lib().moe_linear_backward(R, M, dt, act, dy, z, dz, db, ws, n, None)


@pytest.mark.parametrize("fn,kw,status", [
    (lin, dict(R=-1), INV), (lin, dict(K=0), INV), (lin, dict(M=0), INV), (lin, dict(K=96), UNS), (lin, dict(M=12), UNS),
    (lin, dict(K=(1 << 22) + 64), UNS), (lin, dict(M=(1 << 22) + 8), UNS), (lin, dict(K=1 << 22, M=512), UNS),
    (lin, dict(R=1 << 31), UNS), (lin, dict(R=I63), UNS), (lin, dict(R=1 << 30, M=1024), UNS), (lin, dict(dt=3), INV),
    (lin, dict(act=5), INV), (lin, dict(act=-1), INV), (lin, dict(x=None), INV), (lin, dict(w=None), INV),
    (lin, dict(y=None), INV), (lin, dict(y=p(0)), INV), (lin, dict(y=p(1)), INV), (lin, dict(y=p(2)), INV),
    (lin, dict(y=p(4)), INV), (lin, dict(z=p(3)), INV), (lin, dict(z=p(0)), INV), (lin, dict(b=ODD), INV),
    (lin, dict(R=40, ws=None), WS), (lin, dict(R=40, n=1024), WS), (lin, dict(R=40, ws=ctypes.c_void_p(24)), WS),
    (lin, dict(R=0, x=None, ws=None), OK), (lin, dict(dt=moe.MOE_F32, R=(1 << 31) - 1, M=504), UNS),
    (lin_bwd, dict(R=-1), INV), (lin_bwd, dict(M=4), UNS), (lin_bwd, dict(act=9), INV), (lin_bwd, dict(dy=None), INV),
    (lin_bwd, dict(z=None), INV), (lin_bwd, dict(dz=None, db=None), INV), (lin_bwd, dict(db=ODD), INV),
    (lin_bwd, dict(ws=None), WS), (lin_bwd, dict(n=511), WS),
    (lin_bwd, dict(R=0, db=None), OK), (lin_bwd, dict(R=0, dy=None, z=None, dz=None, db=None, ws=None), OK),
])
def test_linear_errors(fn, kw, status):
    assert fn(**kw) == status


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("K,M", [(64, 8), (1024, 136), (12288, 5120), (256, 65536)])
def test_linear_workspace_never_falls(K, M, dtype):
    sizes = np.array([moe.moe_linear_workspace_size(r, K, M, dtype) for r in range(0, 3000)], np.int64)
    assert (np.diff(sizes) >= 0).all() and sizes[0] == 0
    assert moe.moe_linear_workspace_size((1 << 31) - 1, K, 8, dtype) >= moe.moe_linear_workspace_size(3000, K, 8, dtype)
    assert moe.moe_linear_workspace_size(-1, K, M, dtype) == 0 and moe.moe_linear_workspace_size(4, 100, M, dtype) == 0
    back = np.array([moe.moe_linear_backward_workspace_size(r, M, dtype) for r in range(0, 3000)], np.int64)
    assert (np.diff(back) >= 0).all() and back[0] == 0 and back[1] >= 4 * M


@pytest.mark.parametrize("D", [8, 520, 4096, 16384])
def test_layer_norm_workspace_never_falls(D):
    sizes = np.array([moe.moe_layer_norm_workspace_size(n, D) for n in range(0, 3000)], np.int64)
    assert (np.diff(sizes) >= 0).all() and sizes[0] == 0 and sizes[1] >= 8 * D
    assert moe.moe_layer_norm_workspace_size(-1, D) == 0 and moe.moe_layer_norm_workspace_size(4, D + 4) == 0


CFG = moe.make_config(64, 16, 1, 1, 4, 64)
WIDE = moe.make_config(64, 512, 1, 1, 32, 64)


def bal(cfg=CFG, N=40, T=40, weight=0.1, s=p(0), idx=p(1), mask=p(2), counts=p(3), coef=p(4), loss=p(5), ws=p(6), n=BIG):
    return moe.lib().moe_balance_loss(ctypes.byref(cfg), N, T, weight, s, idx, mask, counts, coef, loss, ws, n, None)


def back(cfg=CFG, N=40, s=p(0), idx=p(1), dw=p(2), T=40, coef=p(3), dloss=p(4), mask=p(5), out=p(6)):
    return moe.lib().moe_route_backward(ctypes.byref(cfg), N, s, idx, dw, T, coef, dloss, mask, out, None)


BAD = moe.make_config(64, 10, 4, 2, 2, 64)


@pytest.mark.parametrize("fn,kw,status", [
    (bal, dict(cfg=BAD), INV), (bal, dict(N=-1), INV), (bal, dict(T=0), INV), (bal, dict(T=-5), INV), (bal, dict(N=1 << 29), UNS),
    (bal, dict(N=I63), UNS), (bal, dict(cfg=WIDE, N=1 << 26), UNS), (bal, dict(N=1 << 27, T=1), UNS),
    (bal, dict(weight=NAN), INV), (bal, dict(weight=INF), INV), (bal, dict(s=None), INV), (bal, dict(idx=None), INV),
    (bal, dict(loss=None), INV), (bal, dict(coef=p(5)), INV), (bal, dict(counts=p(4)), INV), (bal, dict(coef=p(0)), INV),
    (bal, dict(counts=p(1)), INV), (bal, dict(s=ODD), INV), (bal, dict(N=4000, T=4000, ws=None), WS),
    (bal, dict(N=4000, T=4000, n=16), WS), (bal, dict(T=1, ws=None), WS),
    (back, dict(cfg=BAD), INV), (back, dict(N=-1), INV), (back, dict(T=0), INV), (back, dict(N=1 << 29), UNS),
    (back, dict(dw=None, coef=None), INV), (back, dict(idx=None), INV), (back, dict(s=None), INV), (back, dict(out=None), INV),
    (back, dict(out=p(2)), INV), (back, dict(out=p(3)), INV), (back, dict(out=ODD), INV), (back, dict(N=0, s=None), OK),
    (back, dict(N=0, dw=None, coef=None, idx=None, s=None, out=None), OK),
    (back, dict(cfg=WIDE, N=1 << 26), UNS),
])
def test_balance_errors(fn, kw, status):
    assert fn(**kw) == status


@pytest.mark.parametrize("T", [1, 100, 512, 513, 700, 1024, 5000, 100000, 1 << 40])
def test_balance_workspace_never_falls(T):
    for cfg in (CFG, WIDE):
        n = np.unique(np.concatenate([np.arange(0, 2000), 2.0 ** np.arange(11, 22, 0.01)]).astype(np.int64))
        sizes = np.array([moe.moe_balance_workspace_size(cfg, int(i), T) for i in n], np.int64)
        assert (np.diff(sizes) >= 0).all() and sizes[0] == 0


def tensors(*t):
    return (moe.MoeTensor * max(1, len(t)))(*(moe.MoeTensor(a, n, d) for a, n, d in t))


def norm(ts, n=None, out=p(0), ws=p(1), size=BIG):
    return moe.lib().moe_grad_norm(tensors(*ts), len(ts) if n is None else n, out, ws, size, None)


def clip(ts, out=None, n=None, norm=p(1 << 20), m=1.0, eps=1e-6):
    return moe.lib().moe_grad_clip(tensors(*ts), None if out is None else tensors(*out), len(ts) if n is None else n, norm, m, eps,
                                   None)


F, B = moe.MOE_F32, moe.MOE_BF16


def test_tensor_list_workspace_of_any_alignment():
    """A workspace sized for a list serves the same lengths elsewhere."""
    size = moe.lib().moe_grad_norm_workspace_size
    lengths = [2048 * 700, 1, 2047, 2049, 16384 * 40]
    for dt, step in ((F, 4), (B, 2)):
        for scale in (1, 16):
            at = [size(tensors(*((1 << 30 | (off + 8 * i) * step, scale * n, dt) for i, n in enumerate(lengths))), len(lengths))
                  for off in (0, 1, 31, 63)]
            assert len(set(at)) == 1


@pytest.mark.parametrize("fn,args,kw,status", [
    (norm, [[(4096, -1, F)]], {}, INV), (norm, [[(4096, 4, 2)]], {}, INV), (norm, [[(None, 4, F)]], {}, INV),
    (norm, [[(4098, 4, F)]], {}, INV), (norm, [[(4097, 4, B)]], {}, INV), (norm, [[(4096, 1 << 41, B)]], {}, UNS),
    (norm, [[(4096, 1 << 40, B), (1 << 50, 4, B)]], {}, UNS), (norm, [[(4096, I63, B), (4096, I63, B)]], {}, UNS),
    (norm, [[(4096, 4, F)]], dict(n=-1), INV), (norm, [[(4096, 4, F)]], dict(n=65537), UNS),
    (norm, [[(4096, 4, F)]], dict(out=None), INV), (norm, [[(4096, 4, F)]], dict(ws=None), WS),
    (norm, [[(4096, 4, F)]], dict(size=8), WS), (norm, [[(4096, 4, F)]], dict(ws=ctypes.c_void_p(24)), WS),
    (clip, [[(4096, 4, F)]], dict(norm=None), INV), (clip, [[(4096, 4, F)]], dict(m=-1.0), INV),
    (clip, [[(4096, 4, F)]], dict(m=INF), INV), (clip, [[(4096, 4, F)]], dict(eps=NAN), INV),
    (clip, [[(4096, 4, F)]], dict(out=[(8192, 5, F)]), INV), (clip, [[(4096, 4, F)]], dict(out=[(None, 4, F)]), INV),
    # the same tensor twice, two that overlap, in any order; an output over another tensor, or over its own in another type
    (clip, [[(4096, 4, F), (4096, 4, F)]], {}, INV), (clip, [[(8192, 9, F), (4096, 2048, B), (8190, 2, B)]], {}, INV),
    (clip, [[(4096, 4, F), (8192, 4, F)]], dict(out=[(8192, 4, F), (4096, 4, F)]), INV),
    (clip, [[(4096, 4, F), (8192, 4, F)]], dict(out=[(1 << 20, 4, F), (1 << 20, 4, F)]), INV),
    (clip, [[(4096, 4, F)]], dict(out=[(4096, 4, B)]), INV), (clip, [[(4096, 4, F)]], dict(out=[(4100, 4, F)]), INV),
    (clip, [[(1 << 20, 4, B), (4096, 4, F)]], dict(out=[((1 << 20) + 2, 4, B), (4096, 4, F)]), INV),
    # the norm in a tensor that is written, its first and last value and one that half covers it; beside it and in one only read
    (clip, [[(4096, 4, F)]], dict(norm=ctypes.c_void_p(4096)), INV), (clip, [[(4096, 4, F)]], dict(norm=ctypes.c_void_p(4108)), INV),
    (clip, [[(4098, 4, B)]], dict(norm=ctypes.c_void_p(4096)), INV),
    (clip, [[(1 << 20, 4, F)]], dict(out=[(4096, 4, B)], norm=ctypes.c_void_p(4100)), INV),
    (clip, [[]], {}, OK), (clip, [[(None, 0, F), (None, 0, B)]], {}, OK),
])
def test_tensor_list_errors(fn, args, kw, status):
    assert fn(*args, **kw) == status


def test_binding_refuses_host_tensors_and_wrong_types():
    t = torch.zeros(4, 64)
    with pytest.raises(TypeError):
        moe.moe_layer_norm(4, t, None, None, None, None, t)
    with pytest.raises(TypeError):
        moe.moe_linear(t, t, t)
    with pytest.raises(TypeError):
        moe.moe_linear_backward(t, t, t, None)
    for y in (None, t[0], 3):
        with pytest.raises((TypeError, ValueError)):
            moe.moe_linear(t, t, y)
    with pytest.raises(TypeError):
        moe.moe_balance_loss(CFG, 4, t, t, 4, 0.1, None, None, t, None)
    with pytest.raises(TypeError):
        moe.moe_route_backward(CFG, 4, t, t, t, t)
    with pytest.raises(TypeError):
        moe.moe_grad_norm([t], t, None)
    with pytest.raises(TypeError):
        moe.moe_tensor_list([t.half()])
    with pytest.raises(ValueError):
        moe._activation("tanh")
