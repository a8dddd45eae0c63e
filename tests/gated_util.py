"""Plain 64-bit forms of the gated block and of the optimizer step, and the error each result may carry.

The gated product.  z's bound E is product64's (linear_util).  With a = act(g), h = a u: the errors of g and u give
SLOPE E_g (|u| + E_u) + |a| E_u, the activation its own (|v| + 4) 2^-24 |a u| (linear_util), the product one rounding.

sigma = p = 1 / (1 + e), e = 2^(-v log2 e): the argument's roundings are at most (|v| + 1) 2^-22 of e, 2^x, the sum and 1/x
one ulp (2^-23) each.  dp / p = -(1 - p) de / e, so p's relative error is at most r = (1 - p) (|v| + 2) 2^-22 + 2^-21 and
1 - p is off by at most p r + 2^-24.  slope = p + w (1 - p) with w = c p v'(c) (c = g, v' = 1 for SiLU), w off by
(r + 2^-21) |w|: E_slope = p r + |w| ((1 - p) (r + 2^-21) + p r + 2^-24) + 2^-23 (p + |w|).  A p below 2^-126 may come
out as 0 (2^x overflows from x = 128 on, and the hardware's 1 / x gives no subnormal numbers): 2^-126 more of error in p,
so 2^-126 |g| in the activation and 2^-126 (1 + |c v'|) in the slope.

Coded groups.  The scale is amax / 448: off by E_amax / 448 and two roundings.  A code's value times the scale is off
by E and by half a step of E4M3: 2^-4 of the value (normal codes) or 2^-10 of the scale (subnormal ones), where the
quotient's own rounding can move a value across a midpoint: (1 + 2^-20) of that.
"""

import math

import torch

from tests.linear_util import SLOPE, act64, argument, blocks64, rows64

E4M3 = torch.float8_e4m3fn


def gated64(qa, sa, qb, sb, act):
    """(z, E_z, h, E_h) in 64 bits; qb [2n, k]."""
    a, b = rows64(qa, sa), blocks64(qb, sb)
    z, mag = a @ b.t(), a.abs() @ b.abs().t()
    ez = (2.0 ** -10 + (qa.shape[1] // 128 + 2) * 2.0 ** -24) * mag
    n = z.shape[1] // 2
    g, u, eg, eu = z[:, :n], z[:, n:], ez[:, :n], ez[:, n:]
    h = act64(g, act) * u
    eh = SLOPE * eg * (u.abs() + eu) + act64(g, act).abs() * eu + (argument(g, act) + 5) * 2.0 ** -24 * h.abs()
    return z, ez, h, eh


def sigma64(g, act):
    """(p, v, c, v'(c)) of act(g) = g p."""
    if act == "silu":
        return torch.sigmoid(g), g, g, torch.ones_like(g)
    c, k = g.clamp(-16, 16), 2 * math.sqrt(2 / math.pi)
    v = k * (c + 0.044715 * c ** 3)
    return torch.sigmoid(v), v, c, k * (1 + 3 * 0.044715 * c * c)


def backward64(dh, z, act):
    """{name: (value, bound)} of dg, du, h from bf16 dh [m, n], z [m, 2n]."""
    n = dh.shape[1]
    d, g, u = dh.double(), z[:, :n].double(), z[:, n:].double()
    if act in ("relu", "none"):
        a = g.clamp(min=0) if act == "relu" else g
        slope = (g > 0).double() if act == "relu" else torch.ones_like(g)
        ea, es = torch.zeros_like(g), torch.zeros_like(g)
    else:
        p, v, c, dv = sigma64(g, act)
        r = (1 - p) * (v.abs().clamp(max=104) + 2) * 2.0 ** -22 + 2.0 ** -21
        w = c * p * dv
        a, slope = g * p, p + w * (1 - p)
        ea = a.abs() * (r + 2.0 ** -24) + 2.0 ** -126 * g.abs()
        es = 2.0 ** -126 * (1 + (c * dv).abs()) + p * r + w.abs() * ((1 - p) * (r + 2.0 ** -21) + p * r + 2.0 ** -24) + 2.0 ** -23 * (p + w.abs())
    f = 2.0 ** -22
    return {"dg": (d * u * slope, (d * u).abs() * (es + f * slope.abs())),
            "du": (d * a, d.abs() * (ea + f * a.abs())),
            "h": (a * u, u.abs() * (ea + f * a.abs()))}


def check_codes(q, s, want, slack, label):
    """Codes q (uint8 [rows, cols]) and scales [rows, cols/128] of `want` (64 bits) known to within `slack`."""
    q, s, want, slack = q.cpu(), s.cpu().double(), want.cpu(), slack.cpu()
    rows, cols = want.shape
    value = q.view(E4M3).double()
    assert torch.isfinite(value).all() and torch.isfinite(s).all(), f"{label}: not finite"
    top = want.abs().view(rows, -1, 128).amax(2)
    off = slack.view(rows, -1, 128).amax(2)
    allow = (off + 2.0 ** -22 * (top + off)) / 448 + 2.0 ** -149
    worst = float(((s - top / 448).abs() / allow).max()) if top.numel() else 0.0
    assert worst <= 1.0, f"{label}: scales at {worst:.3f} of their bound"
    spread = s.repeat_interleave(128, 1)
    step = torch.maximum(2.0 ** -4 * (want.abs() + slack), 2.0 ** -10 * spread) * (1 + 2.0 ** -20)
    worst = float(((value * spread - want).abs() / (slack + step + 2.0 ** -140)).max()) if want.numel() else 0.0
    assert worst <= 1.0, f"{label}: codes at {worst:.3f} of their bound"


# ---- the optimizer ------------------------------------------------------------------------------


def mix32(x):
    """The library's 32-bit mixing, on int64 tensors."""
    x = x ^ (x >> 16)
    x = (x * 0xBB67AE85) & 0xFFFFFFFF
    x = x ^ (x >> 15)
    x = (x * 0x6A09E667) & 0xFFFFFFFF
    return x ^ (x >> 16)


def random20(seed, step, number, n):
    key = mix32(torch.tensor([(seed + step * 0x9E3779B1) & 0xFFFFFFFF]))
    key = mix32((key + number * 0x3C6EF373) & 0xFFFFFFFF)
    return mix32((key + torch.arange(n) * 0x9E3779B1) & 0xFFFFFFFF) >> 12


def adamw64(p, g, m, v, lr, step, beta1, beta2, eps, decay, grad_scale=1.0):
    """(p, m, v, bounds of the three) in 64 bits from FP32 values; every product, sum, quotient and root of the FP32
    step rounds once (2^-24), hyperparameters too."""
    p, g, m, v = (x.double() for x in (p, g, m, v))
    g = g * grad_scale
    em = 5 * 2.0 ** -24 * ((beta1 * m).abs() + ((1 - beta1) * g).abs())
    ev = 6 * 2.0 ** -24 * (beta2 * v + (1 - beta2) * g * g)
    m, v = beta1 * m + (1 - beta1) * g, beta2 * v + (1 - beta2) * g * g
    b1, b2 = 1 - beta1 ** step, 1 - beta2 ** step
    den = (v / b2).sqrt() + eps
    move = m / b1 / den
    # bias corrections from a step on the device: ln(beta) * step rounds to 2^-23 of itself, expm1 to 2 ulp
    rel = 16 * 2.0 ** -24
    ep = lr * (em / b1 / den + rel * move.abs() + 2.0 ** -21 * abs(decay) * p.abs()) + 2.0 ** -23 * (p.abs() + lr * move.abs())
    return p - lr * (move + decay * p), m, v, ep, em + 1e-45, ev + 1e-45


def check_root_codes(q, s, r, er, bits, label):
    """Codes of r >= 0 (64 bits, within er) rounded at random with these 20 bits, against their scales."""
    n = r.numel()
    pad = (-n) % 128
    top = torch.cat([r, r.new_zeros(pad)]).view(-1, 128).amax(1)
    off = torch.cat([er, r.new_zeros(pad)]).view(-1, 128).amax(1)
    s = s.cpu().double()
    assert float(((s - top / 448).abs() / ((off + 2.0 ** -22 * top) / 448 + 2.0 ** -149)).max()) <= 1.0, f"{label}: scales"
    spread = s.repeat_interleave(128)[:n]
    got = q.cpu().view(E4M3).double().view(-1)
    at = torch.where(spread > 0, r / spread, torch.zeros_like(r)).clamp(max=448)
    step = torch.exp2(torch.floor(torch.log2(at.clamp(min=2.0 ** -6))) - 3)
    t = at / step + bits.double() * 2.0 ** -20
    want = torch.where(r > 0, (torch.floor(t) * step).clamp(2.0 ** -9, 448), torch.zeros_like(r))
    # the quotient is off by its root's, its scale's and its own rounding: 2^-21 of at most 16 steps and of er
    near = (t - t.round()).abs() <= 16 * 2.0 ** -21 + torch.where(spread > 0, er / spread / step, torch.zeros_like(r))
    assert bool((got[r > 0] > 0).all()), f"{label}: a positive value became zero"
    wrong = (got != want) & ~near
    assert not bool(wrong.any()), f"{label}: {int(wrong.sum())} codes, first at {int(wrong.nonzero()[0])}"
    assert bool(((got - want).abs() <= step * 2)[near].all()), f"{label}: a code beyond its neighbour"
