"""The sizes of the GPU tests of the ragged operators reach the kernels that they are meant to reach on 256 CUs."""

from tests.ragged_rules import grouped_tile_rows
from tests.test_gpu_ragged_heights import HEIGHTS, segments


def test_every_tile_height_is_reached():
    for experts, low, high, n, height in HEIGHTS:
        rows = int(segments(experts, low, high)[1][-1])
        assert [grouped_tile_rows(rows, experts, n, b) for b in (0, 1)] == [height, height]
    assert sorted(h[-1] for h in HEIGHTS) == [16, 64, 128, 192, 256]
