"""The sizes of the GPU tests of the ragged operators reach the kernels that they are meant to reach on 256 CUs."""

from tests.ragged_rules import grouped_tile_rows, wgrad_parts
from tests.test_gpu_ragged_heights import HEIGHTS, segments
from tests.test_gpu_wgrad_parts import CASES


def test_every_tile_height_is_reached():
    for experts, low, high, n, height in HEIGHTS:
        rows = int(segments(experts, low, high)[1][-1])
        assert [grouped_tile_rows(rows, experts, n, b) for b in (0, 1)] == [height, height]
    assert sorted(h[-1] for h in HEIGHTS) == [16, 64, 128, 192, 256]


def test_the_rows_are_split_and_unevenly():
    for lengths, m, n, parts in CASES:
        assert wgrad_parts(sum(lengths), len(lengths), m, n) == parts > 1
    slabs = [(-(-rows // 64), parts) for lengths, _, _, parts in CASES for rows in lengths]
    assert any(s == 0 for s, _ in slabs) and any(0 < s < p for s, p in slabs) and any(s > p and s % p for s, p in slabs)
