"""Edges of the operators of a training step on the GPU, against float64 references and exact whole-number results."""
import pytest
import torch

import sparse_moe_layer_gate_amd as moe
from tests import _train as R
from tests._ops import check

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


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
