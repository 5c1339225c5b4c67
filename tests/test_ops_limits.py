"""The largest calls of the operators around the experts: what a launch cannot hold (2^32 threads) and sizes whose
products pass 64 bits are refused on the host, before anything is launched."""
import ctypes

import pytest

import sparse_moe_layer_gate_amd as moe

UNS = moe.MOE_ERR_UNSUPPORTED
BIG = 1 << 60
I63 = (1 << 63) - 1


def p(i):
    return ctypes.c_void_p(4096 * (i + 1))  # never dereferenced


def norm(N, D):
    return moe.lib().moe_block_norm(N, D, moe.MOE_BF16, 1e-5, 1.0, p(0), None, None, None, 0, p(1), None, p(2), None)


def norm_bwd(N, D):
    return moe.lib().moe_block_norm_backward(N, D, moe.MOE_BF16, 1e-5, 1.0, p(0), None, None, None, 0, p(1), None, p(2),
                                             p(3), None, None, None, p(4), p(5), BIG, None)


def combine(N, k, D, R=8):
    return moe.lib().moe_combine(N, k, D, moe.MOE_BF16, p(0), R, p(1), p(2), p(3), 1.0, p(4), None)


def combine_bwd(N, k, D, R=8):
    return moe.lib().moe_combine_backward(N, k, D, moe.MOE_BF16, p(0), p(1), R, p(2), p(3), 1.0, p(4), p(5), None)


@pytest.mark.parametrize("N,D", [(1 << 26, 64), (1 << 22, 8192), (1 << 22, 16384), (5592406, 6144), (1 << 31, 64), (I63, 64)])
def test_norm_rows(N, D):
    """64, 1024, 1024 and 768 threads a row."""
    assert norm(N, D) == UNS


@pytest.mark.parametrize("N", [1 << 31, 1 << 62, I63])
def test_norm_backward_rows(N):
    assert norm_bwd(N, 64) == UNS


@pytest.mark.parametrize("fn", [combine, combine_bwd])
@pytest.mark.parametrize("N,k,D", [(1 << 26, 1, 64), (1 << 22, 1, 8192), (1 << 22, 1, 65536), (1 << 31, 1, 64), (1 << 30, 2, 64),
                                   (1 << 59, 32, 64), (1 << 62, 4, 64), (I63, 2, 64), (I63, 32, 64)])
def test_combine_rows(fn, N, k, D):
    """N k passes 64 bits in the last four."""
    assert fn(N, k, D) == UNS


@pytest.mark.parametrize("rows,K", [(1 << 23, 4096), ((1 << 29) - 31, 64), (1 << 39, 1 << 30), (1 << 36, 1 << 30), (I63, 64)])
def test_quantize_values(rows, K):
    """2^32 pieces of eight values; one more than whole blocks of them leave room for; products past 64 bits."""
    assert moe.lib().moe_quantize(moe.MOE_BF16, rows, K, 32, p(0), p(1), p(2), None) == UNS


def test_grouped_tiles():
    L, wide, R = moe.lib(), 1 << 22, 1 << 20
    for dt, r, E in ((moe.MOE_F32, R, 512), (moe.MOE_F32, R, 1), (moe.MOE_BF16, 512 * 11, 512), (moe.MOE_BF16, 2047, 512)):
        assert L.moe_grouped_linear(E, r, 64, wide, dt, p(0), r, None, 1, p(1), p(2), p(3), p(4), BIG, None) == UNS, (dt, r, E)
    for E in (1, 512):
        assert L.moe_grouped_linear_dgrad(E, R, wide, 64, moe.MOE_F32, p(0), p(1), p(2), p(3), p(4), BIG, None) == UNS
    assert L.moe_grouped_linear_wgrad(512, R, wide, 128, moe.MOE_F32, p(0), p(1), R, None, 1, p(2), p(3), p(4), BIG, None) == UNS


def test_layer_tokens():
    """The layer's own calls: N (k + 1) may not pass 64 bits either."""
    cfg = moe.make_config(256, 16, 4, 2, 3, 128)
    for N in (1 << 62, I63):
        assert moe.moe_workspace_size(cfg, N) == 0
        assert moe.lib().moe_dispatch(ctypes.byref(cfg), N, p(0), p(1), p(2), p(3), p(4), p(5), BIG, None) == UNS


@pytest.mark.gpu
def test_largest_launches():
    """Just below the limit of narrow rows (64 threads each): every row as in a call of 4,096 of them."""
    import torch

    n, D, bf = 4096, 64, dict(dtype=torch.bfloat16, device="cuda")
    N = (1 << 26) - n
    g = torch.Generator(device="cuda").manual_seed(41)
    base = torch.randn((n, D), generator=g, device="cuda").to(torch.bfloat16)
    w, small = torch.ones(D, **bf), torch.empty((n, D), **bf)
    big = base.repeat(N // n, 1)
    out = torch.empty((N, D), **bf)
    moe.moe_block_norm(n, base, None, None, None, 0, w, None, small)
    moe.moe_block_norm(N, big, None, None, None, 0, w, None, out)
    assert (out.view(N // n, n, D) == small).all()
    del big
    inv = torch.arange(n, dtype=torch.int32, device="cuda").flip(0).repeat(N // n)
    moe.moe_combine(N, 1, base, inv, None, None, out, alpha=2.0)
    assert (out.view(N // n, n, D) == 2.0 * base.flip(0)).all()
