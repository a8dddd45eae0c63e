"""Gated products over expert offsets of which some segment runs backwards, by every kernel."""

import pytest
import torch

from tests.gated_rules import kernel
from tests.gated_util import check_codes, gated64
from tests.linear_util import blocks, check, gen, normal, row_tiles

pytestmark = pytest.mark.gpu
NAN = float("nan")

# offsets, of which some segment runs backwards, in units of `unit` rows (no more rows in all segments than there are); rows
BACKWARDS = [([0, 5, 10, 6], 10), ([5, 3, 10], 12), ([4, 5, 0, 1], 12), ([0, 3, 3, 9, 7, 8], 12), ([12, 7, 9, 2, 5, 1], 12),
             ([-4, 2, 2, 30, 30, 0], 12)]
UNITS = {0: (2, 256, 640), 128: (40, 640, 2048), 256: (5, 256, 256)}


@pytest.mark.parametrize("which", sorted(UNITS))
@pytest.mark.parametrize("offsets,rows", BACKWARDS)
def test_segments_that_run_backwards(gpu_lib, which, offsets, rows):
    """Offsets are clipped and a segment that runs backwards is empty, whichever kernel runs: rows of one segment have
    their results in every output, rows of none keep what they held (rows of several have one of their results)."""
    unit, n, k = UNITS[which]
    rows, experts = rows * unit, len(offsets) - 1
    assert kernel(rows, n, k, True, experts) == which
    seg = [min(max(o * unit, 0), rows) for o in offsets]
    owners = torch.zeros(rows, dtype=torch.int64)
    for a, b in zip(seg, seg[1:]):
        owners[a:max(a, b)] += 1
    g = gen(rows + len(offsets))
    qa, sa = row_tiles(normal(g, rows, k))
    qb, sb = blocks(normal(g, experts, 2 * n, k) * 0.05)
    z = torch.full((rows, 2 * n), NAN, dtype=torch.bfloat16, device="cuda")
    h = torch.full((rows, n), NAN, dtype=torch.bfloat16, device="cuda")
    q = torch.full((rows, n), 0x5A, dtype=torch.uint8, device="cuda")
    s = torch.full((rows, n // 128), NAN, device="cuda")
    device_seg = torch.tensor([o * unit for o in offsets], dtype=torch.int32).cuda()
    gpu_lib.fp8bs_grouped_gemm_gated_ragged(qa.cuda(), sa.cuda(), device_seg, qb.cuda(), sb.cuda(), z=z, h=h, qh=q, sh=s)
    torch.cuda.synchronize()
    none = (owners == 0).cuda()
    assert z[none].isnan().all() and h[none].isnan().all() and s[none].isnan().all() and (q[none] == 0x5A).all()
    for e, (a, b) in enumerate(zip(seg, seg[1:])):
        at = torch.arange(a, max(a, b))
        at = at[owners[at] == 1]
        if at.numel():
            z64, ez, h64, eh = gated64(qa[at], sa[at], qb[e], sb[e], "silu")
            check(z[at.cuda()], z64, ez, f"z of {e}")
            check(h[at.cuda()], h64, eh, f"h of {e}")
            check_codes(q[at.cuda()], s[at.cuda()], h64, eh, f"codes of {e}")


@pytest.mark.parametrize("which,rows,k", [(0, 20, 1024), (128, 150, 2048), (256, 100, 128)])
def test_many_experts_of_which_some_run_backwards(gpu_lib, which, rows, k):
    """More experts than a workgroup has threads; the last offset is the first one, so no row lies between the two."""
    experts, n = 300, 128
    assert kernel(rows, n, k, True, experts) == which
    g = gen(which)
    seg = torch.sort(torch.randint(0, rows + 1, (experts + 1,), generator=g)).values
    seg[0], seg[-2], seg[-1] = 0, rows, 0
    qa, sa = row_tiles(normal(g, rows, k))
    qb, sb = blocks(normal(g, 1, 2 * n, k) * 0.05)
    dev = [t.cuda() for t in (qa, sa, seg.int())]
    weights = qb.cuda().expand(experts, -1, -1).contiguous(), sb.cuda().expand(experts, -1, -1).contiguous()
    h, q, s = gpu_lib.fp8bs_grouped_gemm_gated_ragged(*dev, *weights, qh=None)
    torch.cuda.synchronize()
    _, _, h64, eh = gated64(qa, sa, qb[0], sb[0], "silu")
    check(h, h64, eh, "h")
    check_codes(q, s, h64, eh, "codes")
