"""4-bit products beside large activations: the sums are those of x (q - 8), so a weight of 0 (q = 8) adds nothing
whatever its activation, and the error of a row is that of float32 sums of the products themselves."""
import pytest
import torch

import sparse_moe_layer_gate_amd as moe
from tests import _ops as O

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
FORMS = ["16 rows", "32 rows", "64 rows", "48 rows", "experts", "experts few"]


def dev(t):
    return None if t is None else t.cuda()


def case(form, group, seed):
    """x, q, s, the rows' sources and the call's lists, of sizes that run the named form."""
    counts, M = {"16 rows": ([5], 192), "32 rows": ([40], 16384), "64 rows": ([150], 16384), "48 rows": ([390], 5120),
                 "experts": ([0, 1, 15, 31, 33, 47, 49, 64, 65, 129] * 4, 1280), "experts few": ([0, 3, 1, 9] * 16, 256)}[form]
    E, R, K = len(counts), sum(counts), 384
    g = torch.Generator().manual_seed(seed)
    offsets = torch.tensor([0] + counts, dtype=torch.int32).cumsum(0).to(torch.int32)
    index = torch.randperm(R, generator=g).to(torch.int32) if E > 1 else None
    x = torch.randn((R, K), generator=g).to(BF)
    q = torch.randint(0, 256, (E, M, K // 2), generator=g, dtype=torch.uint8)
    s = (torch.rand((E, M, K // group), generator=g) + 0.5).mul(0.01).to(BF)
    return offsets, index, x, q, s


def product(offsets, index, x, q, s):
    R = x.shape[0]
    y = torch.full((R, q.shape[1]), 7.0, dtype=BF, device="cuda")
    kw = dict(offsets=dev(offsets), row_index=dev(index)) if index is not None else {}
    moe.moe_qlinear(dev(x), dev(q), dev(s), y, **kw)
    torch.cuda.synchronize()
    return y.cpu()


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("form", FORMS)
def test_zero_weights_add_nothing(form, group):
    """Two features whose weights are all 0: their activations, up to bfloat16's largest, leave every bit as it is."""
    print(f"[zero weights] {form} group={group}", flush=True)
    offsets, index, x, q, s = case(form, group, 31)
    q[..., 50 // 2] = (q[..., 50 // 2] & 0xf0) | 8    # feature 50 (low half)
    q[..., 301 // 2] = (q[..., 301 // 2] & 0x0f) | 0x80  # feature 301 (high half)
    out = []
    for big in (0.0, 2.0 ** 20, -float(torch.finfo(BF).max)):
        x[:, 50], x[:, 301] = big, big
        out.append(product(offsets, index, x, q, s))
    assert torch.isfinite(out[0].float()).all()
    assert torch.equal(out[0], out[1]) and torch.equal(out[0], out[2])


@pytest.mark.parametrize("outlier", [1.0, 1e4, 1e6])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("form", FORMS)
def test_error_of_float32_sums(form, group, outlier):
    """One feature's activations `outlier` times the others'. Bound: a group's float32 sum (one step of 2^-23 per term,
    if the matrix core's additions are cut rather than rounded), its scaling, and the sum over the groups, each of the
    products' magnitudes; then the output's rounding."""
    print(f"[outliers] {form} group={group} outlier={outlier}", flush=True)
    offsets, index, x, q, s = case(form, group, 32)
    x[:, 77] = (x[:, 77].float() * outlier).to(BF)
    K = x.shape[1]
    y = product(offsets, index, x, q, s)
    w = O.dequantize(q, s)
    src = index.long() if index is not None else torch.arange(x.shape[0])
    ref = O.grouped(x.double(), w, offsets, src, x.shape[0])
    mag = O.grouped(x.double().abs(), w.abs(), offsets, src, x.shape[0])
    O.check("y", y, ref, (2 * group + K / group + 4) * O.U32 * mag)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_quantize_shows_nan_and_infinity(group, dtype):
    """A NaN (of either sign, at any place of the group) or an infinity becomes the group's scale; the other groups are
    quantised as without it, and a product shows it in the rows of that weight alone."""
    K, rows = 512, 64
    g = torch.Generator().manual_seed(33)
    w = torch.randn((1, rows, K), generator=g).to(dtype)
    clean_q, clean_s = moe.moe_quantize(dev(w), group)
    bad = w.clone()
    inf, nan = float("inf"), float("nan")
    at = {3: (0, nan), 10: (group - 1, -nan), 20: (group // 2, inf), 33: (7, -inf), 40: (5, nan), 41: (1, inf)}
    for row, (k, v) in at.items():
        bad[0, row, group + k] = v        # the row's second group
    bad[0, 40, group + 6] = inf           # beside a NaN
    bad[0, 41, group:2 * group] = inf     # nothing else
    q, s = moe.moe_quantize(dev(bad), group)
    sc, qc = s.cpu().float()[0], q.cpu()[0]
    for row, (_, v) in at.items():
        assert (sc[row, 1].isnan() if v != v else sc[row, 1] == inf), (row, sc[row, 1])
        assert (qc[row, group // 2:group] == 0x88).all(), row
    same_s, same_q = s.clone(), q.clone()
    for row in at:
        same_s[0, row, 1] = clean_s[0, row, 1]
        same_q[0, row, group // 2:group] = clean_q[0, row, group // 2:group]
    assert torch.equal(same_s, clean_s) and torch.equal(same_q, clean_q)
    x = torch.randn((3, K), generator=g).to(BF)
    y, ref = (torch.empty((3, rows), dtype=BF, device="cuda") for _ in range(2))
    moe.moe_qlinear(dev(x), q, s, y)
    moe.moe_qlinear(dev(x), clean_q, clean_s, ref)
    hit = torch.zeros(rows, dtype=torch.bool)
    hit[list(at)] = True
    assert y.cpu()[:, hit].isnan().all()
    assert torch.equal(y.cpu()[:, ~hit], ref.cpu()[:, ~hit])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize_group_whose_scale_vanishes(dtype):
    """Magnitudes so small that a seventh of them rounds to 0 in bfloat16: scale 0, q = 8."""
    w = torch.full((2, 64), float(torch.finfo(torch.bfloat16).smallest_normal) / 128, dtype=dtype)  # the least bfloat16
    q, s = moe.moe_quantize(dev(w), 32)
    assert (s.cpu() == 0).all() and (q.cpu() == 0x88).all()


@pytest.mark.parametrize("limit", [0.0, 1.5])
@pytest.mark.parametrize("form", ["16 rows", "64 rows", "experts"])
def test_swiglu_shows_nan(form, limit):
    """NaN scales of one gate row and one up row, and a NaN activation row: their outputs and no others are NaN, clamped
    or not."""
    offsets, index, x, q, s = case(form, 64, 34)
    M = q.shape[1] // 128 * 128
    q, s = q[:, :M].contiguous(), s[:, :M].contiguous()
    half = M // 2
    kw = dict(offsets=dev(offsets), row_index=dev(index)) if index is not None else {}

    def run():
        y = torch.full((x.shape[0], half), 7.0, dtype=BF, device="cuda")
        moe.moe_qlinear(dev(x), dev(q), dev(s), y, swiglu=True, limit=limit, **kw)
        return y.cpu()
    clean = run()
    s[:, 5, 1] = float("nan")
    s[:, half + 9, 0] = float("nan")
    x[2, 17] = float("nan")
    y = run()
    row = int((index == 2).nonzero()[0, 0]) if index is not None else 2
    hit = torch.zeros_like(y, dtype=torch.bool)
    hit[:, 5] = hit[:, 9] = True
    hit[row] = True
    assert torch.isfinite(clean.float()).all() and y[hit].isnan().all()
    assert torch.equal(y[~hit], clean[~hit])
