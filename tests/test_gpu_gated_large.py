"""Gated products whose outputs pass the caches."""

import pytest
import torch

from tests.gated_rules import kernel
from tests.linear_util import blocks, gen, normal, row_tiles

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("experts", [0, 3])
def test_large_outputs_have_the_bits_of_their_parts(gpu_lib, experts):
    """bf16 outputs beyond 128 MiB pass the caches: the same bits as calls on a third of the rows each."""
    m, n, k = 3 * 3840, 2048, 256
    part = m // 3
    assert m * n * 6 > 128 << 20 > part * n * 6
    assert {kernel(m, n, k, True, experts), kernel(part, n, k, True, 1 if experts else 0)} == {256}
    g = gen(m)
    qa, sa = (t.cuda() for t in row_tiles(normal(g, m, k)))
    qb, sb = (t.cuda() for t in blocks(normal(g, max(1, experts), 2 * n, k) * 0.05))
    z = torch.empty((m, 2 * n), dtype=torch.bfloat16, device="cuda")

    def call(rows, e, z):
        a, b = qa[rows], sa[rows]
        if not experts:
            return gpu_lib.fp8bs_gemm_gated(a, b, qb[0], sb[0], z=z, qh=None)
        seg = torch.tensor([0, part, 2 * part, m] if e is None else [0, part], dtype=torch.int32, device="cuda")
        w = slice(None) if e is None else slice(e, e + 1)
        return gpu_lib.fp8bs_grouped_gemm_gated_ragged(a, b, seg, qb[w], sb[w], z=z, qh=None)

    whole = (z, *call(slice(None), None, z))
    for e in range(3):
        rows = slice(e * part, (e + 1) * part)
        zp = torch.empty((part, 2 * n), dtype=torch.bfloat16, device="cuda")
        for a, b in zip(whole, (zp, *call(rows, e, zp))):
            assert torch.equal(a[rows].view(torch.uint8), b.view(torch.uint8))
