"""Size limits of the gated backward pass, at their edges: host checks, no kernel is launched (a pointer is misaligned, so
that a call whose sizes pass ends there)."""

import pytest

from tests.test_gated_args import BWD, EALIGN, ESHAPE, NONE, OK, P, call


@pytest.fixture(scope="module")
def lib():
    from fp8_fine_grained_act_amd import lib

    return lib


@pytest.mark.parametrize("pieces", [1, 3, 1000, (1 << 23) - 1])
def test_backward_rows_limit(lib, pieces):
    """m ceil(n / 128) < 2^31 - 16."""
    n, most = 128 * pieces, ((1 << 31) - 17) // pieces
    wide = dict(NONE, dz=P, n=n, lddh=n, ldz=2 * n, lddz=2 * n, dh=P + 8)
    f = lib.raw.fp8bs_gated_backward
    assert call(f, BWD, **dict(wide, m=most)) == EALIGN
    assert call(f, BWD, **dict(wide, m=most + 1)) == ESHAPE
    assert call(f, BWD, **dict(wide, m=0, dh=P)) == OK
    assert call(f, BWD, **dict(wide, m=0, dh=P, n=n - 120, lddh=n, ldz=2 * n)) == OK


def test_backward_width_limit(lib):
    n = 1 << 30
    wide = dict(NONE, dz=P, m=1, lddh=n, ldz=2 * n, lddz=2 * n, dh=P + 8)
    assert call(lib.raw.fp8bs_gated_backward, BWD, **dict(wide, n=n)) == ESHAPE
    assert call(lib.raw.fp8bs_gated_backward, BWD, **dict(wide, n=n - 8)) == EALIGN
