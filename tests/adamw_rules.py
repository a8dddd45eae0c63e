"""The optimizer step with states in 8 bits, restated in single FP32 operations on the host, random bits included."""

import torch

from tests.gated_util import E4M3, mix32

F = lambda x: torch.tensor(x, dtype=torch.float32)  # noqa: E731


def words(seed, step, number, n):
    """The 32 random bits of each element: their upper 20 round sqrt(v), the upper 20 of their mix round m."""
    key = mix32(torch.tensor([(seed + step * 0x9E3779B1) & 0xFFFFFFFF]))
    key = mix32((key + number * 0x3C6EF373) & 0xFFFFFFFF)
    return mix32((key + torch.arange(n) * 0x9E3779B1) & 0xFFFFFFFF)


def at_random(q, bits):
    """q in [0, 448] to the E4M3 value below or above, by 20 random bits below the last kept one."""
    move = torch.where(q < 2.0 ** -6, 2.0 ** -6, 0.0)
    x = ((q + move).view(torch.int32).long() + bits) & ~0xFFFFF
    return x.to(torch.int32).view(torch.float32) - move


def held(beta1):
    """Codes below this are those that rounding to nearest may hold while there is no gradient: at most 0.5 / (1 - beta1)
    units; the subnormal ones have up to 7, all others 8 to 15."""
    return float("inf") if (1 - beta1) * 8 < 0.5 else 2.0 ** -6


class States8:
    """m and sqrt(v) of n elements (a multiple of 128) as codes and scales.  nearest: m always to nearest."""

    def __init__(self, n, nearest=False):
        self.m, self.r = torch.zeros(n), torch.zeros(n)           # code values
        self.ms, self.rs = torch.zeros(n // 128), torch.zeros(n // 128)
        self.nearest = nearest

    def step(self, g, step, beta1, beta2, seed=0, number=0):
        """New states; returns m and sqrt(v) before they are rounded, from which the update is made."""
        spread = lambda s: s.repeat_interleave(128)  # noqa: E731
        m = self.m * spread(self.ms) * F(beta1) + g * F(1 - beta1)
        r = self.r * spread(self.rs)
        r = ((r * r) * F(beta2) + (g * g) * F(1 - beta2)).double().sqrt().float()   # FP32's on the host is not to nearest
        word = words(seed, step, number, g.numel())
        scales = [x.abs().view(-1, 128).amax(1) * F(1 / 448) for x in (m, r)]
        q = [torch.where(spread(s) > 0, x / spread(s), 0 * x).clamp(-448, 448) for x, s in zip((m, r), scales)]
        code = q[0].to(E4M3).float()
        if not self.nearest:
            top = torch.where(spread(self.ms) > 0, torch.maximum(self.m.abs(), q[0].abs()), float("inf"))
            by_chance = torch.copysign(at_random(q[0].abs(), mix32((word + 0x3C6EF373) & 0xFFFFFFFF) >> 12), q[0])
            code = torch.where(top < held(beta1), by_chance, code)
        self.m, self.ms, self.rs = code, scales[0], scales[1]
        self.r = torch.where(r > 0, at_random(q[1], word >> 12).clamp(2.0 ** -9, 448), 0.0)
        return m, r


def update(m, r, step, beta1, beta2, eps=1e-8):
    """What a step subtracts, in units of lr."""
    m, r = m.double(), r.double()
    return m / (1 - beta1 ** step) / (r / (1 - beta2 ** step) ** 0.5 + eps)
