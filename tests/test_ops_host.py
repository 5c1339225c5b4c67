"""The operators around the experts without a GPU: argument errors are found on the host before any launch,
sizes never fall, and the Python binding refuses tensors that are not on a device."""
import ctypes

import numpy as np
import pytest

import sparse_moe_layer_gate_amd as moe

INV, UNS, WS, OK = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED, moe.MOE_ERR_WORKSPACE, moe.MOE_OK
BIG = 1 << 40


def p(i):
    return ctypes.c_void_p(4096 * (i + 1))  # never dereferenced


def norm(N=4, D=256, dt=moe.MOE_BF16, eps=1e-5, a=1.0, h=p(0), o=p(1), w_post=p(2), gate=p(3), T=2, w_pre=p(4),
         h_out=p(5), u=p(6)):
    return moe.lib().moe_block_norm(N, D, dt, eps, a, h, o, w_post, gate, T, w_pre, h_out, u, None)


def norm_bwd(N=4, D=256, dt=moe.MOE_BF16, eps=1e-5, a=1.0, h_out=p(0), o=p(1), w_post=p(2), gate=p(3), T=2, w_pre=p(4),
             dh_out=p(5), du=p(6), dh=p(7), d_o=p(8), dwp=p(9), dg=p(10), dw=p(11), ws=p(12), n=BIG):
    return moe.lib().moe_block_norm_backward(N, D, dt, eps, a, h_out, o, w_post, gate, T, w_pre, dh_out, du, dh, d_o,
                                             dwp, dg, dw, ws, n, None)


@pytest.mark.parametrize("kw,status", [
    (dict(N=-1), INV), (dict(D=0), INV), (dict(D=200), UNS), (dict(D=16448), UNS), (dict(N=1 << 31), UNS),
    (dict(dt=2), INV), (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV), (dict(a=float("inf")), INV),
    (dict(T=0), INV), (dict(h=None), INV), (dict(h_out=None), INV), (dict(u=None), INV), (dict(w_pre=None), INV),
    (dict(o=None), INV),                                   # gate, w_post and h_out belong to o
    (dict(o=None, w_post=None, gate=None), INV),           # h_out does too
    (dict(o=None, w_post=None, gate=None, h_out=None, w_pre=None, u=None), INV),  # nothing to do
    (dict(u=p(0)), INV), (dict(u=p(5)), INV), (dict(h_out=p(1)), INV), (dict(h=ctypes.c_void_p(4100)), INV),
    (dict(N=0, h=None), OK),
])
def test_block_norm_errors(kw, status):
    assert norm(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(N=-1), INV), (dict(D=96), UNS), (dict(T=0), INV), (dict(h_out=None), INV), (dict(dh=None), INV),
    (dict(d_o=None), INV), (dict(dh_out=None, du=None), INV), (dict(du=None), INV), (dict(w_pre=None), INV),
    (dict(w_post=None), INV), (dict(gate=None), INV), (dict(o=None), INV), (dict(dh=p(0)), INV), (dict(d_o=p(7)), INV),
    (dict(d_o=p(5)), INV), (dict(ws=None), WS), (dict(n=1024), WS), (dict(ws=ctypes.c_void_p(8)), WS),
])
def test_block_norm_backward_errors(kw, status):
    assert norm_bwd(**kw) == status


@pytest.mark.parametrize("T", [0, 1, 7, 512, 1 << 40])
def test_block_norm_workspace_never_falls(T):
    sizes = np.array([moe.moe_block_norm_workspace_size(n, 512, "bf16", T) for n in range(0, 4000)], np.int64)
    assert (np.diff(sizes) >= 0).all() and sizes[0] == 0 and sizes[1] >= 2 * 512 * 4
    assert moe.moe_block_norm_workspace_size(-1, 512) == 0 and moe.moe_block_norm_workspace_size(4, 100) == 0


def combine(N=4, k=2, D=256, dt=moe.MOE_BF16, rows=p(0), R=8, inv=p(1), w=p(2), sh=p(3), alpha=1.0, y=p(4)):
    return moe.lib().moe_combine(N, k, D, dt, rows, R, inv, w, sh, alpha, y, None)


def combine_bwd(N=4, k=2, D=256, dt=moe.MOE_BF16, dy=p(0), rows=p(1), R=8, inv=p(2), w=p(3), alpha=1.0, drows=p(4),
                dw=p(5)):
    return moe.lib().moe_combine_backward(N, k, D, dt, dy, rows, R, inv, w, alpha, drows, dw, None)


@pytest.mark.parametrize("fn,kw,status", [
    (combine, dict(N=-1), INV), (combine, dict(k=0), INV), (combine, dict(k=33), UNS), (combine, dict(D=100), UNS),
    (combine, dict(R=-1), INV), (combine, dict(N=1 << 30, k=4), UNS), (combine, dict(alpha=float("nan")), INV),
    (combine, dict(rows=None), INV), (combine, dict(inv=None), INV), (combine, dict(y=None), INV),
    (combine, dict(y=p(0)), INV), (combine, dict(dt=7), INV), (combine, dict(N=0, inv=None), OK),
    (combine_bwd, dict(dy=None), INV), (combine_bwd, dict(rows=None), INV), (combine_bwd, dict(w=None), INV),
    (combine_bwd, dict(drows=None), INV), (combine_bwd, dict(drows=p(0)), INV), (combine_bwd, dict(drows=p(1)), INV),
    (combine_bwd, dict(k=40), UNS), (combine_bwd, dict(N=0), OK),
])
def test_combine_errors(fn, kw, status):
    assert fn(**kw) == status


def fwd(E=4, R=8, K=256, M=128, dt=moe.MOE_BF16, x=p(0), xr=8, idx=None, div=1, w=p(1), off=p(2), y=p(3), ws=p(4), n=BIG):
    return moe.lib().moe_grouped_linear(E, R, K, M, dt, x, xr, idx, div, w, off, y, ws, n, None)


def dgrad(E=4, R=8, K=256, M=128, dt=moe.MOE_BF16, dy=p(0), w=p(1), off=p(2), dx=p(3), ws=p(4), n=BIG):
    return moe.lib().moe_grouped_linear_dgrad(E, R, K, M, dt, dy, w, off, dx, ws, n, None)


def wgrad(E=4, R=8, K=256, M=128, dt=moe.MOE_BF16, dy=p(0), x=p(1), xr=8, idx=None, div=1, off=p(2), dw=p(3), ws=p(4), n=BIG):
    return moe.lib().moe_grouped_linear_wgrad(E, R, K, M, dt, dy, x, xr, idx, div, off, dw, ws, n, None)


@pytest.mark.parametrize("kw,status", [
    (dict(E=0), INV), (dict(E=513), UNS), (dict(R=-1), INV), (dict(R=1 << 31), UNS), (dict(K=100), UNS),
    (dict(M=96), UNS), (dict(M=0), INV), (dict(dt=2), INV), (dict(K=65536, M=32768), UNS), (dict(off=None), INV),
])
@pytest.mark.parametrize("fn", [fwd, dgrad, wgrad])
def test_grouped_errors(fn, kw, status):
    assert fn(**kw) == status


def test_grouped_source_and_buffers():
    for fn in (fwd, wgrad):
        assert fn(xr=7) == INV                                 # fewer rows than R without an index
        assert fn(idx=p(5), div=0) == INV
        assert fn(idx=p(5), xr=0) == INV
        assert fn(idx=p(5), xr=1 << 31) == UNS
        assert fn(idx=p(5), xr=1 << 30, K=64, M=64) == UNS     # gathered x of 4 GiB and more
        assert fn(idx=p(5), n=64) == WS
        assert fn(idx=p(5), ws=None) == WS
    assert fwd(n=64) == WS and dgrad(n=64) == WS
    assert fwd(y=p(0)) == INV and dgrad(dx=p(0)) == INV and wgrad(dw=p(0)) == INV
    assert fwd(x=None) == INV and dgrad(dy=None) == INV and wgrad(dw=None) == INV
    assert fwd(R=0, x=None, xr=0) == OK and dgrad(R=0, dy=None) == OK


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_grouped_workspace_never_falls(dtype):
    for E in (1, 16, 256, 512):
        sizes = np.array([moe.moe_grouped_workspace_size(E, r, dtype) for r in range(0, 20000, 13)], np.int64)
        assert (np.diff(sizes) >= 0).all()
    assert moe.moe_grouped_workspace_size(513, 4, dtype) == 0 and moe.moe_grouped_workspace_size(4, -1, dtype) == 0


def qlin(E=4, R=8, K=256, M=128, group=64, x=p(0), xr=8, idx=None, div=1, wq=p(1), s=p(2), off=p(3), sw=0, lim=0.0, y=p(4)):
    return moe.lib().moe_qlinear(E, R, K, M, group, x, xr, idx, div, wq, s, off, sw, lim, y, None)


@pytest.mark.parametrize("kw,status", [
    (dict(E=0), INV), (dict(E=513), UNS), (dict(group=0), INV), (dict(group=16), UNS), (dict(group=128, K=320), INV),
    (dict(K=100), UNS), (dict(M=100), UNS), (dict(sw=2), INV), (dict(sw=1, M=192), UNS), (dict(sw=1, lim=-1.0), INV),
    (dict(lim=1.0), INV), (dict(off=None), INV), (dict(xr=4), INV), (dict(idx=p(6), div=0), INV), (dict(x=None), INV),
    (dict(wq=None), INV), (dict(s=None), INV), (dict(y=None), INV), (dict(y=p(0)), INV), (dict(R=-1), INV),
    (dict(R=0, x=None, xr=0), OK), (dict(E=1, R=0, off=None, xr=0), OK),
])
def test_qlinear_errors(kw, status):
    assert qlin(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dt=3), INV), (dict(rows=-1), INV), (dict(group=48), UNS), (dict(group=-1), INV), (dict(K=100, group=32), INV),
    (dict(K=96, group=32), UNS), (dict(w=None), INV), (dict(q=None), INV), (dict(s=None), INV), (dict(q=p(0)), INV),
    (dict(rows=0, w=None), OK),
])
def test_quantize_errors(kw, status):
    a = dict(dt=moe.MOE_BF16, rows=4, K=256, group=64, w=p(0), q=p(1), s=p(2))
    a.update(kw)
    assert moe.lib().moe_quantize(a["dt"], a["rows"], a["K"], a["group"], a["w"], a["q"], a["s"], None) == status


def test_binding_refuses_host_tensors():
    import torch

    h = torch.zeros(4, 64)
    with pytest.raises(TypeError):
        moe.moe_block_norm(4, h, None, None, None, 0, torch.ones(64), None, torch.empty(4, 64))
    with pytest.raises(TypeError):
        moe.moe_grouped_linear(h, torch.zeros(2, 64, 64), torch.zeros(3, dtype=torch.int32), h, None)
    with pytest.raises(TypeError):
        moe.moe_quantize(h.half(), 32)
    with pytest.raises(ValueError):
        moe.moe_quantize(h, 48)
