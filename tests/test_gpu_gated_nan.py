"""Values that are not finite in the gated block's coded outputs: a NaN or an infinity makes its whole tile NaN (the scale
is NaN, as the quantizers make it), whatever stands beside it, and changes nothing else."""

import pytest
import torch

from tests.gated_rules import kernel
from tests.gated_util import E4M3
from tests.linear_util import ACTS, blocks, gen, normal, row_tiles

pytestmark = pytest.mark.gpu
NAN = float("nan")

# rows, n, k that reach each kernel with codes asked for, and the same over segments
DENSE = {0: (7, 256, 640), 128: (700, 384, 1920), 256: (300, 640, 512)}
RAGGED = {0: ([3, 0, 1], 256, 640), 128: ([200, 0, 190, 210], 384, 2048), 256: ([300, 5, 128, 127, 0, 129], 256, 640)}


def tiles(q, s):
    """What the codes stand for, by tile: [rows, tiles, 128]."""
    return q.cpu().view(E4M3).double().view(q.shape[0], -1, 128) * s.cpu().double()[:, :, None]


def same_but(got, clean, bad, label, touched=None):
    """Tiles marked in `bad` [rows, tiles] are NaN as a whole, the others have the bits of the clean call (but for those
    marked in `touched`, whose inputs differ)."""
    bad = bad.cpu()
    assert tiles(*got)[bad].isnan().all(), f"{label}: a tile hides what is not finite"
    bad = bad if touched is None else bad | touched
    q, q0 = (t[0].cpu().view(*bad.shape, 128)[~bad] for t in (got, clean))
    assert torch.equal(q, q0) and torch.equal(got[1].cpu()[~bad], clean[1].cpu()[~bad]), f"{label}: another tile changed"


@pytest.mark.parametrize("which", sorted(DENSE))
@pytest.mark.parametrize("act", ["relu", "gelu_tanh", "silu"])
def test_forward(gpu_lib, which, act):
    m, n, k = DENSE[which]
    assert kernel(m, n, k, True) == which
    g = gen(m)
    qa, sa = row_tiles(normal(g, m, k))
    qb, sb = blocks(normal(g, 2 * n, k) * 0.05)
    qa[1], sa[1] = 0, 0.0                         # a row of zeros beside the one to come
    call = lambda *t: gpu_lib.fp8bs_gemm_gated(*(x.cuda() for x in t), act=ACTS[act], qh=None)  # noqa: E731
    h0, *clean = call(qa, sa, qb, sb)
    for value in (NAN, 3e38):                     # a row of NaN, a row whose pre-activations overflow
        bad_sa = sa.clone()
        bad_sa[2, 0] = value
        h, *got = call(qa, bad_sa, qb, sb)
        bad = (~h.isfinite()).view(m, -1, 128).any(2)
        assert bad[2].all() and not bad[:2].any() and not bad[3:].any()
        same_but(got, clean, bad, f"row of {value}")
        assert torch.equal(h[3:].view(torch.int16), h0[3:].view(torch.int16))
    for at in (5, n + 133):                       # one gate weight, one up weight: a column of NaN
        bad_qb = qb.clone()
        bad_qb[at, 7] = 0x7F
        h, *got = call(qa, sa, bad_qb, sb)
        bad = h.isnan().view(m, -1, 128).any(2)
        assert int(h.isnan().sum()) == m and bad[:, at % n // 128].all()
        same_but(got, clean, bad, f"weight row {at}")


@pytest.mark.parametrize("which", sorted(RAGGED))
def test_segments(gpu_lib, which):
    lengths, n, k = RAGGED[which]
    m, experts = sum(lengths), len(lengths)
    assert kernel(m, n, k, True, experts) == which
    g = gen(n)
    qa, sa = row_tiles(normal(g, m, k))
    qb, sb = blocks(normal(g, experts, 2 * n, k) * 0.05)
    qa[1], sa[1] = 0, 0.0
    seg = torch.tensor([0] + lengths).cumsum(0).int()
    call = lambda a, b: gpu_lib.fp8bs_grouped_gemm_gated_ragged(*(x.cuda() for x in (qa, a, seg, b, sb)), qh=None)  # noqa: E731
    h0, *clean = call(sa, qb)
    bad_sa = sa.clone()
    bad_sa[2] = NAN
    h, *got = call(bad_sa, qb)
    bad = h.isnan().view(m, -1, 128).any(2)
    assert bad[2].all() and int(h.isnan().sum()) == n
    same_but(got, clean, bad, "row")
    bad_qb, last = qb.clone(), max(e for e in range(experts) if lengths[e])
    bad_qb[last, n + 130, 3] = 0x7F
    h, *got = call(sa, bad_qb)
    bad = h.isnan().view(m, -1, 128).any(2)
    assert bad[int(seg[last]):int(seg[last + 1]), 1].all() and int(h.isnan().sum()) == lengths[last]
    same_but(got, clean, bad, "weight row")


@pytest.mark.parametrize("act", ["none", "gelu_tanh", "silu"])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("transposed", [False, True])
def test_backward(gpu_lib, act, zeros, transposed):
    m, n = 256, 384
    g = gen(m + n)
    dh, z = (normal(g, m, n) * 1e-3).bfloat16(), normal(g, m, 2 * n).bfloat16()
    if zeros:                                     # groups of zeros in every wave, along both axes
        dh[::2] = 0.0
        dh[:, ::2] = 0.0
        dh[1, :128] = dh[1, 128:256] = 0.0
        z[:, 10] = 0.0
    more = dict(qt=None, qht=None) if transposed else {}
    call = lambda d, v: gpu_lib.fp8bs_gated_backward(d.cuda(), v.cuda(), act=ACTS[act], q=None, h=None, **more)  # noqa: E731
    clean = call(dh, z)
    spots = {"dh": (37, 130), "up": (137, 5), "gate": (200, 383)}
    for name, (r, c) in spots.items():
        for value in (NAN, float("inf")):
            d, v = dh.clone(), z.clone()
            d[r, c] = 1.0 if name != "dh" else value
            if name == "up":
                v[r, n + c] = value
            elif name == "gate":
                v[r, c] = value
            base = call(torch.where(torch.isfinite(d), d, 0.0), torch.where(torch.isfinite(v), v, 0.0))
            dz, q, s, qt, st, h, qht, sht = call(d, v)
            off = ~dz.isfinite()
            assert off.any() and int(off.sum()) <= 2 and int((~h.isfinite()).sum()) <= 1
            label = f"{value} in {name}"
            spot = torch.zeros(m, 2 * n, dtype=torch.bool)
            spot[r, [c, n + c]] = True
            rows = lambda t: t.view(m, -1, 128).any(2)  # noqa: E731
            cols = lambda t: t.t().reshape(t.shape[1], -1, 128).any(2)  # noqa: E731
            same_but((q, s), (base[1], base[2]), rows(off), f"{label}: q", rows(spot))
            if transposed:
                same_but((qt, st), (base[3], base[4]), cols(off), f"{label}: qt", cols(spot))
                same_but((qht, sht), (base[6], base[7]), cols(~h.isfinite()), f"{label}: qht", cols(spot[:, :n]))
    d = dh.clone()
    d[99] = NAN                                   # a row as a whole
    dz, q, s, qt, st, *_ = call(d, z)
    bad = torch.zeros(m, 2 * n // 128, dtype=torch.bool)
    bad[99] = True
    same_but((q, s), (clean[1], clean[2]), bad, "row: q")
    if transposed:
        bad = torch.zeros(2 * n, m // 128, dtype=torch.bool)
        bad[:, 0] = True
        same_but((qt, st), (clean[3], clean[4]), bad, "row: qt")
