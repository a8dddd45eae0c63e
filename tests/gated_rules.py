"""The host rule by which a gated product chooses its kernel (gated_tile_cols), restated for 256 CUs, so that a test can
say which kernel its sizes reach: 0 for the few-row tiles, 128 or 256 for the weight rows of a large tile."""

import math

CUS = 256
ROW_SHAPES = ((1, 1, 7), (1, 2, 11), (2, 2, 16), (2, 4, 21))


def few_row_shape(rows, experts, n):
    """(cost, (row groups, column groups)) of the cheapest few-row tile; experts 0: one weight."""
    def tiles(bm):
        return (rows + (bm - 1) * min(experts, rows)) // bm if experts else -(-rows // bm)
    return min((-(-tiles(16 * mt) * (n // (8 * nt)) // CUS) * cost, i, (mt, nt))
               for i, (mt, nt, cost) in enumerate(ROW_SHAPES))[::2]


def kernel(rows, n, k, codes, experts=0):
    owners = min(experts, rows) if experts else 1
    mean = rows / owners
    high = mean + 2.0 * math.sqrt(mean) if owners > 1 else mean
    full = math.floor(high / 128)
    rest = high - 128 * full
    cost_of = lambda r, bn: {128: 21.0, 256: 36.0}[bn] if r <= 64 else {128: 30.0, 256: 50.0}[bn]  # noqa: E731
    extra = (2.5 + 1.8e-6 * rows * n) * 56 * 128 / k if codes else 0.0
    best, best_cost = 0, few_row_shape(rows, experts, n)[0] + extra
    for bn in (128, 256):
        strips = owners * (n // (bn // 2))
        one = cost_of(128 if full else rest, bn)
        total = full * cost_of(128, bn) + (cost_of(rest, bn) if rest > 0 else 0.0)
        tiles = full + (rest > 0)
        cost = max(one, strips * total / CUS) if experts else one * math.ceil(strips * tiles / CUS)
        cost += extra if bn == 128 else 0.0
        if cost < best_cost:
            best, best_cost = bn, cost
    return best
