"""Every tile height of fp8bs_grouped_gemm_ragged: long contractions, and what a value that is not a number may reach."""

import numpy as np
import pytest
import torch

from tests.linear_util import blocks, check, product64, row_tiles
from tests.ragged_rules import CUS, grouped_tile_rows

pytestmark = pytest.mark.gpu

# (experts, fewest rows, most rows, n) -> tile rows of both layouts
HEIGHTS = [(5, 0, 6, 256, 16), (64, 0, 8, 2048, 64), (64, 40, 80, 1024, 128), (64, 100, 150, 1024, 192),
           (64, 190, 256, 1024, 256)]


def segments(experts, low, high):
    lengths = [int(v) for v in np.random.default_rng(low + high).integers(low, high + 1, experts)]
    lengths[1], lengths[-1] = 0, high
    return lengths, torch.tensor([0] + list(np.cumsum(lengths)), dtype=torch.int32)


def on_cus():
    return torch.cuda.get_device_properties(0).multi_processor_count == CUS


def operands(seed, rows, e, n, k, b_layout):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    qa, sa = row_tiles(torch.randn((rows, k), generator=g, device="cuda"))
    qb, sb = blocks(torch.randn((e, n, k) if b_layout == 0 else (e, k, n), generator=g, device="cuda") * 0.05)
    # scales that differ from block to block by up to 16 times: another block's scale cannot pass for the right one
    for s in (sa, sb):
        s.mul_(0.25 + 3.75 * torch.rand(s.shape, generator=g, device="cuda"))
    return qa, sa, qb, sb


@pytest.mark.parametrize("b_layout", [0, 1])
@pytest.mark.parametrize("experts,low,high,n,height", HEIGHTS)
def test_not_a_number_stays_one(gpu_lib, experts, low, high, n, height, b_layout):
    """A scale that is NaN, with the payload that an integer rounding carries into the sign, makes its row or its
    expert's 128 columns NaN, and changes nothing else."""
    k = 384
    lengths, seg = segments(experts, low, high)
    rows = int(seg[-1])
    assert not on_cus() or grouped_tile_rows(rows, experts, n, b_layout) == height
    qa, sa, qb, sb = operands(high + b_layout, rows, experts, n, k, b_layout)
    seg_d = seg.cuda()
    clean = gpu_lib.fp8bs_grouped_gemm_ragged(qa, sa, seg_d, qb, sb, b_layout=b_layout)
    nan = torch.tensor([0x7FFFFFFF], dtype=torch.int32, device="cuda").view(torch.float32)[0]
    want = torch.zeros((rows, n), dtype=torch.bool)
    bad_rows = [0, rows // 2, rows - 1]
    for i, r in enumerate(bad_rows):
        sa[r, i] = nan
        want[r] = True
    e, part = experts - 1, n // 128 - 1                               # the last expert has `high` rows
    (sb[e, part] if b_layout == 0 else sb[e, :, part])[1] = nan
    want[int(seg[e]):int(seg[e + 1]), 128 * part:128 * part + 128] = True
    got = gpu_lib.fp8bs_grouped_gemm_ragged(qa, sa, seg_d, qb, sb, b_layout=b_layout)
    torch.cuda.synchronize()
    assert torch.isfinite(clean).all()
    got, clean = got.cpu(), clean.cpu()
    assert torch.equal(torch.isnan(got), want)
    assert torch.equal(got[~want].view(torch.int16), clean[~want].view(torch.int16))


@pytest.mark.parametrize("blocks_k", [1, 2, 13])
@pytest.mark.parametrize("b_layout", [0, 1])
@pytest.mark.parametrize("experts,low,high,n,height", HEIGHTS)
def test_short_and_long_contractions(gpu_lib, experts, low, high, n, height, b_layout, blocks_k):
    """13 blocks: every stage of a ring is refilled several times, the row scales are fetched for four blocks at a
    time into both their buffers, and the last fetch is for one block.  1 and 2: the ring is not even filled."""
    k = 128 * blocks_k
    lengths, seg = segments(experts, low, high)
    rows = int(seg[-1])
    assert not on_cus() or grouped_tile_rows(rows, experts, n, b_layout) == height
    qa, sa, qb, sb = operands(3 * high + b_layout, rows, experts, n, k, b_layout)
    c = torch.full((rows + 2, n + 8), 9.0, dtype=torch.bfloat16, device="cuda")
    gpu_lib.fp8bs_grouped_gemm_ragged(qa, sa, seg.cuda(), qb, sb, b_layout=b_layout, c=c[:rows, :n])
    torch.cuda.synchronize()
    assert (c[rows:] == 9.0).all() and (c[:, n:] == 9.0).all()
    for i, length in enumerate(lengths):
        cut = slice(int(seg[i]), int(seg[i + 1]))
        if length:
            y, err = product64(qa[cut], sa[cut], qb[i], sb[i], b_layout)
            check(c[cut, :n], y.cpu(), err.cpu(), f"expert {i}, {length} rows")
