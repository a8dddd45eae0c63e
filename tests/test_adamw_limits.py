"""Numbers that the optimizer step refuses: host checks, no kernel is launched (a pointer is misaligned, so that a call
whose numbers pass ends there)."""

import pytest

from tests.test_gated_args import EALIGN, EFLAG, P, STEP, entry


@pytest.fixture(scope="module")
def lib():
    from fp8_fine_grained_act_amd import lib

    return lib


@pytest.mark.parametrize("eps,ok", [(0.0, True), (2.0 ** -126, True), (1e-8, True), (1e-38, False), (1e-45, False), (1e-300, False),
                                    (float("inf"), True)])
def test_eps_that_fp32_cannot_divide_by(lib, eps, ok):
    """1 / eps overflows below 2^-126, and 0 / eps would be NaN for a weight that never had a gradient."""
    table = (lib._AdamwTensor * 1)(entry(lib, param=P + 4))
    assert lib.raw.fp8bs_adamw_step(table, 1, *dict(STEP, eps=eps).values()) == (EALIGN if ok else EFLAG)
