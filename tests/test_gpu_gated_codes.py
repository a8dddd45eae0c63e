"""Codes of the gated backward pass, bit by bit where the coded values are known to the bit."""

import pytest
import torch

from tests.gated_util import E4M3
from tests.linear_util import ACTS, gen, normal

pytestmark = pytest.mark.gpu


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
