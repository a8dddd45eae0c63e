"""States in 8 bits over many steps, by their rule (adamw_rules) against FP32 states."""

import pytest
import torch

from tests.adamw_rules import States8, update
from tests.linear_util import gen

BETA2, N = 0.95, 128 * 8
COLUMN = torch.arange(N) % 128


@pytest.fixture(autouse=True)
def one_thread():
    """The tensors are small: threads only wait for each other."""
    threads = torch.get_num_threads()
    torch.set_num_threads(1)
    yield
    torch.set_num_threads(threads)


def rest_steps(beta1):
    """Steps after which m of at most 448 units has come to zero, but for one element in 10^13: its expected size falls
    by beta1 a step, and below one unit that is the chance that it is not zero."""
    return int(40 / (1 - beta1))


def run(beta1, gradient, first, last, nearest=False):
    """The movement of each weight over steps first + 1 .. last in units of lr: (states in 8 bits, in FP32), and the 8-bit states."""
    s, m, v = States8(N, nearest), torch.zeros(N, dtype=torch.float64), torch.zeros(N, dtype=torch.float64)
    moved = torch.zeros(2, N, dtype=torch.float64)
    for step in range(1, last + 1):
        g = gradient(step)
        m8, r8 = s.step(g, step, beta1, BETA2)
        m, v = beta1 * m + (1 - beta1) * g.double(), BETA2 * v + (1 - BETA2) * g.double() ** 2
        if step > first:
            moved[0] += update(m8, r8, step, beta1, BETA2)
            moved[1] += update(m, v.sqrt(), step, beta1, BETA2)
    return moved, s


def falling_silent(scale):
    """Noise, and from step 101 on `scale` of it in one column of eight."""
    g = gen(7)
    return lambda step: torch.randn(N, generator=g) * 1e-3 * torch.where((COLUMN % 8 == 3) & (step > 100), scale, 1.0)


@pytest.mark.parametrize("beta1", [0.9, 0.93, 0.95, 0.99])
def test_weights_without_a_gradient_come_to_rest(beta1):
    quiet = 100 + rest_steps(beta1)
    moved, s = run(beta1, falling_silent(0.0), quiet, quiet + 100)
    silent = COLUMN % 8 == 3
    assert not s.m[silent].any() and not moved[0][silent].any()
    assert (moved[0][~silent] != 0).all()


def test_rounding_to_nearest_would_keep_them_moving():
    moved, s = run(0.9, falling_silent(0.0), 600, 700, nearest=True)
    silent = COLUMN % 8 == 3
    assert (s.m[silent] != 0).float().mean() > 0.5 and moved[0][silent].abs().mean() > 10


@pytest.mark.parametrize("beta1", [0.9, 0.95])
def test_weights_of_a_negligible_gradient_slow_down(beta1):
    """The gradient is below the group's range: sqrt(v) rests on its smallest code, so the update is smaller than with
    FP32 states but for what random rounding adds: steps of one code's size both ways.  Held codes would add 0.1 a step."""
    moved, _ = run(beta1, falling_silent(1e-6), 1000, 2000)
    silent = COLUMN % 8 == 3
    assert moved[0][silent].abs().mean() / 1000 < 0.03


@pytest.mark.parametrize("beta1", [0.9, 0.95, 0.99])
def test_one_live_weight_in_a_group(beta1):
    """One steady gradient keeps the group's scale; the others have 20 steps of 0.02 of it, then none."""
    gradient = lambda step: torch.where(COLUMN == 0, 1.0, 0.02 if step <= 20 else 0.0)  # noqa: E731
    quiet = 20 + rest_steps(beta1)
    moved, _ = run(beta1, gradient, quiet, quiet + 100)
    assert not moved[0][COLUMN > 0].any()
    # m and sqrt(v) of the steady one are the group's largest, code 448 at every step: the two roundings of each scale
    assert (moved[0][COLUMN == 0] / 100 - 1).abs().max() < 1e-4


@pytest.mark.parametrize("beta1", [0.95, 0.99])
def test_a_steady_gradient_after_a_larger_one(beta1):
    """Where nearest could hold any code, m at random nears the gradient without bias.  sqrt(v) carries the variance of
    its own rounding, at most (1/8)^2 / 4 of its square a step over 1 / (1 - beta2) steps: 8% of a bias in its inverse."""
    gradient = lambda step: torch.where(COLUMN == 0, 1.0, 0.02 if step <= 20 else 0.001)  # noqa: E731
    quiet = 20 + rest_steps(beta1)
    moved, _ = run(beta1, gradient, quiet, quiet + 400)
    mean = moved[:, COLUMN > 0].mean(1) / 400
    assert (mean[0] - mean[1]).abs() < 0.1 and (mean[1] - 1).abs() < 1e-3
