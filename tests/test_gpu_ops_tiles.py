"""The grouped bf16 products when a persistent block gets several tiles: at most one block per CU runs, so calls with
more than twice as many tiles as the card has CUs make every block pass from tile to tile with loads and stores in
flight. Integer operands, so every output is the exact value rounded once (tests/_ops.py)."""
import pytest
import torch

import sparse_moe_layer_gate_amd as moe
from tests import _ops as O

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def dev(t):
    return None if t is None else t.cuda()


def cus():
    return torch.cuda.get_device_properties(0).multi_processor_count


def offsets_of(counts):
    return torch.tensor([0] + counts, dtype=torch.int32).cumsum(0).to(torch.int32)


def workspace(E, R):
    n = moe.moe_grouped_workspace_size(E, R)
    return torch.empty(max(n, 256), dtype=torch.uint8, device="cuda").fill_(0xFF)


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("K,M", [(1344, 1088), (1088, 1344), (1280, 1024)])
def test_wgrad_stream_over_tile_borders(K, M, gather):
    """About 700 tiles: a block's second and third tiles have one to 33 steps of 32 rows, so a tile's stores are in
    flight while the next tile's counted waits run, behind and before experts without rows and of one step, with edge
    rows and columns (waves whose rows lie past the matrix store nothing)."""
    counts = [130, 0, 97, 300, 1, 128, 513, 0, 129, 160, 0, 255, 97, 224, 33, 0, 1031, 192, 0, 100, 257, 64, 31, 351,
              0, 0, 96, 99, 352, 5] + ([128, 127, 161, 320, 0, 140] if M == 1024 else [])
    E, R, N = len(counts), sum(counts) + 9, 500
    tiles = E * ((M + 255) // 256) * ((K + 255) // 256)
    assert tiles > 2.5 * cus(), "every block has to get a second tile, most a third"
    print(f"[wgrad borders] K={K} M={M} gather={gather} tiles={tiles}", flush=True)
    g = torch.Generator().manual_seed(21)
    offsets = offsets_of(counts)
    pair = torch.randint(0, 3 * N, (R,), generator=g, dtype=torch.int32)
    x, dy = O.ints(g, (N if gather else R, K), -3, 3), O.ints(g, (R, M), -3, 3)
    for t in (dy,) if gather else (dy, x):  # rows of no expert: none of their values may reach a sum
        t[R - 9:] = float("nan")
    src = (pair // 3).long() if gather else torch.arange(R)
    kw = dict(row_index=dev(pair), index_div=3) if gather else {}
    args = dev(dy), dev(x), dev(offsets)
    ws = workspace(E, R)
    dw = torch.full((E, M, K), 7.0, dtype=BF, device="cuda")
    moe.moe_grouped_linear_wgrad(*args, dw, ws, **kw)
    torch.cuda.synchronize()
    ref = O.grouped_wgrad(dy.double(), x.double(), offsets, src, E).to(BF)
    for e in range(E):
        assert torch.equal(dw[e].cpu(), ref[e]), (e, counts[e])
    again = torch.full_like(dw, 5.0)
    moe.moe_grouped_linear_wgrad(*args, again, ws, **kw)
    assert torch.equal(again, dw)


@pytest.mark.parametrize("M", [64, 128, 192, 832])
def test_forward_and_dgrad_over_tile_borders(M):
    """More than 600 tiles that hold rows: every block claims a second one over the same LDS, with reductions of one,
    two, three and more steps, tiles of every number of live waves and padding tiles between."""
    K = 1344
    counts = [0, 1, 255, 256, 257, 700, 64, 511, 513, 33, 600, 0, 129, 192, 1025, 31] * 3 + [300] * 14
    E, R = len(counts), sum(counts) + 5
    tiles = sum((c + 255) // 256 for c in counts) * ((K + 255) // 256)
    assert tiles > 2.2 * cus(), "every block has to claim a second tile"
    print(f"[dgrad borders] M={M} tiles={tiles}", flush=True)
    g = torch.Generator().manual_seed(22)
    offsets = offsets_of(counts)
    used = int(offsets[-1])
    w, dy = O.ints(g, (E, M, K), -3, 3), O.ints(g, (R, M), -3, 3)
    ws, o = workspace(E, R), dev(offsets)
    dx = torch.full((R, K), 7.0, dtype=BF, device="cuda")
    moe.moe_grouped_linear_dgrad(dev(dy), dev(w), o, dx, ws)
    torch.cuda.synchronize()
    ref = O.grouped_dgrad(dy.double(), w.double(), offsets)[:used].to(BF)
    assert torch.equal(dx[:used].cpu(), ref)
    assert (dx[used:] == 7.0).all()
    wt = w.transpose(1, 2).contiguous()  # the same product as a forward: K output columns
    y = torch.full((R, K), 7.0, dtype=BF, device="cuda")
    moe.moe_grouped_linear(dev(dy), dev(wt), o, y, ws)
    torch.cuda.synchronize()
    assert torch.equal(y[:used].cpu(), ref)
    assert (y[used:] == 7.0).all()
