"""Codes of the gated backward pass, bit by bit; expert segments that run backwards; large forward calls."""

import pytest
import torch

from tests.gated_rules import kernel
from tests.gated_util import E4M3, check_codes, gated64
from tests.linear_util import ACTS, blocks, check, gen, normal, row_tiles

pytestmark = pytest.mark.gpu
NAN = float("nan")


def nearest_codes(x):
    """Codes and scales of 1x128 tiles of FP32 values: the nearest, ties to even, of the binary32 quotient x / (amax / 448)."""
    t = x.double().view(x.shape[0], -1, 128)
    s = (t.abs().amax(2) / 448).float()
    q = torch.where(s[:, :, None] > 0, t / s[:, :, None].double(), 0 * t).float()
    return q.clamp(-448, 448).to(E4M3).view(torch.uint8).view(x.shape), s


@pytest.mark.parametrize("m,n", [(256, 128), (1024, 1280), (2048, 2048)])
@pytest.mark.parametrize("act", ["none", "relu"])
def test_backward_codes_are_the_nearest(gpu_lib, m, n, act):
    """Without an activation, and with ReLU, dz and h are products of two bf16 values, exact in FP32: the coded values are
    known to the bit.  A quotient of 64 bits rounded to 32 and the kernel's own differ where they meet a rounding boundary
    of binary32 within 2^-46, and a code then only where that is a midpoint of two codes too: never, in a few million."""
    g = gen(m + n)
    dh, z = (normal(g, m, n) * 1e-3).bfloat16(), (normal(g, m, 2 * n) * 1.5).bfloat16()
    d, gate, up = dh.float(), z[:, :n].float(), z[:, n:].float()
    a, slope = (gate.clamp(min=0), (gate > 0).float()) if act == "relu" else (gate, torch.ones_like(gate))
    dz, h = torch.cat([d * up * slope, d * a], 1), a * up
    _, q, s, qt, st, _, qht, sht = gpu_lib.fp8bs_gated_backward(dh.cuda(), z.cuda(), act=ACTS[act], dz=False, q=None, qt=None,
                                                                qht=None)
    _, q1, s1, *_ = gpu_lib.fp8bs_gated_backward(dh.cuda(), z.cuda(), act=ACTS[act], dz=False, q=None)
    for got, scale, x, label in ((q, s, dz, "columns"), (q1, s1, dz, "columns alone"), (qt, st, dz.t().contiguous(), "rows"),
                                 (qht, sht, h.t().contiguous(), "h along the rows")):
        want, want_s = nearest_codes(x)
        assert torch.equal(scale.cpu(), want_s), f"{label}: scales"
        off = (got.cpu() != want) & ((got.cpu() | want) & 0x7F != 0)     # zeros of either sign
        assert not off.any(), f"{label}: {int(off.sum())} of {off.numel()} codes are not the nearest"


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


@pytest.mark.parametrize("experts", [0, 3])
def test_large_outputs_have_the_bits_of_their_parts(gpu_lib, experts):
    """bf16 outputs beyond 128 MiB pass the caches: the same bits as calls on a third of the rows each."""
    m, n, k = 3 * 3840, 2048, 256
    part = m // 3
    assert m * n * 6 > 128 << 20 > part * n * 6
    assert {kernel(m, n, k, True, experts), kernel(part, n, k, True, 1 if experts else 0)} == {256}
    g = gen(m)
    qa, sa = (t.cuda() for t in row_tiles(normal(g, m, k)))
    qb, sb = (t.cuda() for t in blocks(normal(g, max(1, experts), 2 * n, k) * 0.05))
    z = torch.empty((m, 2 * n), dtype=torch.bfloat16, device="cuda")

    def call(rows, e, z):
        a, b = qa[rows], sa[rows]
        if not experts:
            return gpu_lib.fp8bs_gemm_gated(a, b, qb[0], sb[0], z=z, qh=None)
        seg = torch.tensor([0, part, 2 * part, m] if e is None else [0, part], dtype=torch.int32, device="cuda")
        w = slice(None) if e is None else slice(e, e + 1)
        return gpu_lib.fp8bs_grouped_gemm_gated_ragged(a, b, seg, qb[w], sb[w], z=z, qh=None)

    whole = (z, *call(slice(None), None, z))
    for e in range(3):
        rows = slice(e * part, (e + 1) * part)
        zp = torch.empty((part, 2 * n), dtype=torch.bfloat16, device="cuda")
        for a, b in zip(whole, (zp, *call(rows, e, zp))):
            assert torch.equal(a[rows].view(torch.uint8), b.view(torch.uint8))
