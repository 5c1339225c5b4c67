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
