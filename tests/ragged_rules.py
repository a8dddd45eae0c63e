"""The host rules by which the ragged operators choose a tile height or a number of parts, restated for 256 CUs,
so that a test can say which kernel its sizes reach.  fp8bs_grouped_gemm_ragged: skinny_cost and ragged_tile_rows;
fp8bs_grouped_wgrad_ragged: wgrad_splits."""

import math

CUS = 256


def _tiles(rows, experts, bm):
    return (rows + (bm - 1) * min(experts, rows)) // bm


def _skinny_cost(rows, experts, n, b_layout):
    shapes = ((1, 1, 7), (1, 2, 11), (2, 2, 16), (2, 4, 21)) if b_layout == 0 else ((1, 8, 14), (2, 8, 20))
    return min(-(-_tiles(rows, experts, 16 * mt) * (n // (16 * nt)) // CUS) * cost for mt, nt, cost in shapes)


def grouped_tile_rows(rows, experts, n, b_layout):
    """Rows of a tile, 16 standing for every shape of the few-row kernels."""
    if _skinny_cost(rows, experts, n, b_layout) < 23:
        return 16
    owners = min(experts, rows)
    mean = rows / owners
    high = mean if owners == 1 else mean + 2.0 * math.sqrt(mean)
    strips = owners * (n // 128)

    def tile(r):
        return max(11.5, 4.0 + 4.5 * math.ceil(r / 64.0))

    best, best_cost = 64, math.ceil(strips * math.ceil(high / 64.0) / (2.0 * CUS)) * 21.0
    for bm in (128, 192, 256):
        full = math.floor(high / bm)
        rest = high - full * bm
        one = tile(bm) if full else tile(rest)
        cost = max(one, strips * (full * tile(bm) + (tile(rest) if rest > 0 else 0.0)) / CUS)
        if cost < best_cost:
            best, best_cost = bm, cost
    return best


def wgrad_parts(rows, experts, m, n):
    """Parts into which fp8bs_grouped_wgrad_ragged splits the rows (wgrad_splits), 1: not split."""
    tiles = experts * -(-m // 256) * -(-n // 128)
    slabs = rows // (experts * 64)
    if 2 * tiles > CUS or slabs < 48:
        return 1
    return min(CUS // tiles, slabs // 8, 32)
