"""Plain 64-bit forms of the linear-layer and ragged-expert operators, and the error each result may carry.

Bounds.  A product sum_kb sa sb P_kb is allowed E = (2^-10 + (nkb + 2) 2^-24) * mag, mag = sum_kb sa sb sum |a b|:
2^-10 of a block's sum of |products| for the matrix core's own summation (the allowance of gpu_util, four times the
measured worst), one FP32 rounding per block for the running sum and one for each scale product.  The epilogue adds
one rounding for the bias, act at most multiplies an error by its largest slope (1.13 for GELU, 1.10 for SiLU) and
adds (|v| + 4) 2^-24 |z| of its own (v the exponent's argument: one ulp each for 2^x and 1/x, the rounding of the
argument scaled by |v|), the residual one rounding more.  Rounding to bf16 costs at most 2^-8 of the value.
"""

import math

import torch

ACTS = {"none": 0, "relu": 1, "gelu_tanh": 2, "silu": 3}
SLOPE = 1.13


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def normal(g, *shape):
    return torch.randn(shape, generator=g, dtype=torch.float32)


def row_tiles(x):
    """E4M3 codes (uint8) and FP32 scales of 1x128 tiles along the columns."""
    t = x.reshape(x.shape[0], x.shape[1] // 128, 128)
    s = t.abs().amax(2) / 448.0 if t.numel() else t.new_zeros(t.shape[:2])
    q = (t / s.clamp(min=1e-30)[:, :, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return q.view(torch.uint8).reshape(x.shape), s.contiguous()


def blocks(w):
    """Codes and scales of 128x128 blocks (of a matrix or a stack of matrices)."""
    v = w.reshape(*w.shape[:-2], w.shape[-2] // 128, 128, w.shape[-1] // 128, 128)
    s = v.abs().amax((-3, -1)) / 448.0
    q = (v / s[..., :, None, :, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return q.view(torch.uint8).reshape(w.shape), s.contiguous()


def rows64(q, s):
    return q.view(torch.float8_e4m3fn).double() * s.double().repeat_interleave(128, 1)


def blocks64(q, s):
    return q.view(torch.float8_e4m3fn).double() * s.double().repeat_interleave(128, 0).repeat_interleave(128, 1)


def product64(qa, sa, qb, sb, b_layout):
    """(z, its error bound) of the block-scaled product in 64 bits."""
    a, b = rows64(qa, sa), blocks64(qb, sb)
    b = b.t() if b_layout == 0 else b
    mag = a.abs() @ b.abs()
    return a @ b, (2.0 ** -10 + (qa.shape[1] // 128 + 2) * 2.0 ** -24) * mag


def act64(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if act == "silu":
        return z * torch.sigmoid(z)
    return z


def slope64(z, act):
    if act == "relu":
        return (z > 0).double()
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    if act == "silu":
        p = torch.sigmoid(z)
        return p + z * p * (1 - p)
    return torch.ones_like(z)


def argument(z, act):
    """|v| of sigma(v), where sigma is not saturated (beyond |v| = 104 it is 0 or 1 in FP32 too)."""
    if act == "gelu_tanh":
        return (2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)).abs().clamp(max=104)
    return z.abs().clamp(max=104) if act == "silu" else torch.zeros_like(z)


def check(got, want, slack, label, bf16=True):
    """got within slack (plus half a bf16 step of the larger of the two) of the 64-bit result, element by element."""
    got, want = got.detach().cpu().double(), want.double()
    assert got.shape == want.shape, (label, got.shape, want.shape)
    allow = slack + (2.0 ** -8 * (want.abs() + slack) if bf16 else 0.0) + 1e-37
    off = (got - want).abs()
    assert torch.isfinite(got).all(), f"{label}: not finite"
    worst = float((off / allow).max()) if off.numel() else 0.0
    assert worst <= 1.0, f"{label}: {worst:.3f} of the allowed error"
    return worst
