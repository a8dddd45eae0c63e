"""The sizes of the gated block's GPU tests reach every kernel, on 256 CUs, with and without codes."""

from tests.gated_rules import few_row_shape, kernel
from tests.test_gpu_gated import SEGMENTS, SIZES


def test_every_kernel_is_reached():
    dense = {(kernel(m, n, k, codes), codes) for m, n, k, _ in SIZES for codes in (False, True)}
    assert dense == {(b, c) for b in (0, 128, 256) for c in (False, True)}
    ragged = {(kernel(lead + sum(lengths) + tail, n, k, codes, len(lengths)), codes)
              for lengths, n, k, _, lead, tail in SEGMENTS for codes in (False, True)}
    assert ragged == {(b, c) for b in (0, 128, 256) for c in (False, True)}


def test_every_few_row_shape_is_reached():
    assert {few_row_shape(m, 0, n)[1] for m, n, k, _ in SIZES if kernel(m, n, k, False) == 0} == {(1, 1), (1, 2), (2, 2), (2, 4)}
    assert len({few_row_shape(lead + sum(x) + tail, len(x), n)[1] for x, n, k, _, lead, tail in SEGMENTS
                if kernel(lead + sum(x) + tail, n, k, False, len(x)) == 0}) == 4


def test_the_library_chooses_as_restated():
    """Seen from the workspace, which only the widest tiles need none of (256 CUs where there is no GPU)."""
    from fp8_fine_grained_act_amd import lib

    for m in (1, 7, 33, 64, 100, 130, 300, 513, 700, 1037, 2048, 3000, 4099, 20000):
        for n in (128, 256, 640, 1408, 2048, 7168):
            for k in (128, 512, 2048, 7168):
                need = 0 if kernel(m, n, k, True) == 256 else 4 * m * n
                assert lib.raw.fp8bs_gemm_gated_workspace(m, n, k) == need, (m, n, k)
                for e in (1, 3, 40, 256):
                    need = 0 if kernel(m, n, k, True, e) == 256 else 4 * m * n
                    assert lib.raw.fp8bs_grouped_gemm_gated_ragged_workspace(e, m, n, k) == need, (m, n, k, e)
