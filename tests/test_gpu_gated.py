"""The gated block on the GPU against its 64-bit form (gated_util): forward, over expert segments, backward."""

import pytest
import torch

from tests.gated_rules import kernel
from tests.gated_util import E4M3, backward64, check_codes, gated64
from tests.linear_util import ACTS, blocks, check, gen, normal, row_tiles

pytestmark = pytest.mark.gpu
NAN = float("nan")


def operands(g, m, n, k, scale=1.0, spread=True):
    x = normal(g, m, k) * scale
    if spread and k > 128:
        x[:, :: 97] *= 20.0
    qa, sa = row_tiles(x)
    qb, sb = blocks(normal(g, 2 * n, k) * 0.05)
    return qa, sa, qb, sb


def bf16_buffer(rows, cols, stride):
    """A bf16 matrix inside a wider buffer of NaN, one row more below it: (buffer, view)."""
    b = torch.full((rows + 1, stride), NAN, dtype=torch.bfloat16, device="cuda")
    return b, b[:rows, :cols]


def code_buffer(rows, cols, stride):
    b = torch.full((rows + 1, stride), 0x5A, dtype=torch.uint8, device="cuda")
    return b, b[:rows, :cols]


def untouched(buffer, rows, cols, mark):
    mask = torch.ones(buffer.shape, dtype=torch.bool, device="cuda")
    mask[:rows, :cols] = False
    rest = buffer[mask]
    return bool(rest.isnan().all()) if mark != mark else bool((rest == mark).all())


SIZES = [
    (1, 128, 128, "silu"), (4, 2048, 2048, "silu"), (17, 256, 384, "gelu_tanh"), (33, 384, 1280, "relu"), (130, 128, 128, "none"),
    (64, 640, 512, "silu"), (300, 640, 512, "gelu_tanh"), (1037, 1408, 1024, "gelu_tanh"), (2500, 256, 256, "silu"),
    (129, 1280, 1920, "relu"), (3000, 1152, 384, "silu"), (4099, 1024, 128, "none"),
    (32, 4096, 256, "silu"), (300, 2048, 4096, "silu"),
]


@pytest.mark.parametrize("m,n,k,act", SIZES)
def test_forward(gpu_lib, m, n, k, act):
    g = gen(m + n + k)
    host = operands(g, m, n, k)
    dev = [t.cuda() for t in host]
    zb, z = bf16_buffer(m, 2 * n, 2 * n + 16)
    hb, h = bf16_buffer(m, n, n + 24)
    qb, q = code_buffer(m, n, n + 32)
    s = torch.full((m, n // 128), NAN, device="cuda")
    out = gpu_lib.fp8bs_gemm_gated(*dev, act=ACTS[act], z=z, h=h, qh=q, sh=s)
    torch.cuda.synchronize()
    assert out[0] is h and out[1] is q and out[2] is s
    z64, ez, h64, eh = gated64(*host, act)
    check(z, z64, ez, "z")
    check(h, h64, eh, "h")
    check_codes(q, s, h64, eh, "codes")
    assert untouched(zb, m, 2 * n, NAN) and untouched(hb, m, n, NAN) and untouched(qb, m, n, 0x5A)
    # the outputs of a call do not depend on which others it makes, but for codes, which can choose another kernel
    only_h, none_q, none_s = gpu_lib.fp8bs_gemm_gated(*dev, act=ACTS[act])
    assert none_q is None and none_s is None
    check(only_h, h64, eh, "h alone")
    if kernel(m, n, k, False) == kernel(m, n, k, True):
        assert torch.equal(only_h.view(torch.int16), h.contiguous().view(torch.int16))
    none_h, only_q, only_s = gpu_lib.fp8bs_gemm_gated(*dev, act=ACTS[act], h=False, qh=None)
    assert none_h is None and torch.equal(only_q, q) and torch.equal(only_s, s)
    torch.cuda.synchronize()


@pytest.mark.parametrize("m", [5, 700])
def test_forward_of_zeros_and_tiny_values(gpu_lib, m):
    """Rows of zeros: +-0 codes and scale 0.  Values whose groups' scale is subnormal or zero keep their bound."""
    n, k = 128, 256
    qa, sa, qb, sb = operands(gen(m), m, n, k, spread=False)
    qa[1::5] = 0
    sa[1::5] = 0
    for row, factor in ((2, 2.0 ** -40), (3, 2.0 ** -62), (4, 2.0 ** -70)):
        sa[row::5] *= factor                      # h is of the square of that
    dev = [t.cuda() for t in (qa, sa, qb, sb)]
    z = torch.empty((m, 2 * n), dtype=torch.bfloat16, device="cuda")
    h, q, s = gpu_lib.fp8bs_gemm_gated(*dev, act=0, z=z, qh=None)
    torch.cuda.synchronize()
    z64, ez, h64, eh = gated64(qa, sa, qb, sb, "none")
    check(z, z64, ez, "z")
    check(h, h64, eh + 2.0 ** -133, "h")          # bf16's smallest step
    check_codes(q, s, h64, eh + 2.0 ** -149, "codes")
    zero = (q[1::5] & 0x7F).cpu()
    assert not zero.any() and not s[1::5].any()


def segments_case(g, lengths, n, k, lead=0, tail=0):
    """Operands, offsets and rows of segments of these lengths, `lead` rows before the first, `tail` behind the last."""
    e, rows = len(lengths), lead + sum(lengths) + tail
    x = normal(g, rows, k)
    x[:, ::61] *= 10.0
    qa, sa = row_tiles(x)
    qb, sb = blocks(normal(g, e, 2 * n, k) * 0.05)
    seg = [lead]
    for length in lengths:
        seg.append(seg[-1] + length)
    return qa, sa, torch.tensor(seg, dtype=torch.int32), qb, sb


SEGMENTS = [
    ([1], 128, 128, "silu", 0, 0), ([0, 3, 0, 0, 1, 7, 0], 256, 512, "silu", 0, 2), ([1] * 24, 128, 1024, "gelu_tanh", 0, 0),
    ([130, 0, 1, 64, 17], 384, 384, "relu", 5, 9), ([300, 5, 128, 127, 0, 129], 256, 640, "silu", 0, 3),
    ([1000], 128, 256, "none", 3, 1), ([2, 600, 33, 0, 0, 190, 257, 64], 1024, 256, "silu", 1, 70),
    ([0, 0, 0], 128, 128, "silu", 4, 4), ([40] * 30, 640, 128, "gelu_tanh", 0, 0),
    ([200, 0, 190, 210], 1280, 3200, "silu", 2, 2), ([600, 300, 700], 2048, 256, "silu", 0, 1),
    ([2, 1, 0, 3] * 25, 512, 512, "gelu_tanh", 0, 0),
]


@pytest.mark.parametrize("lengths,n,k,act,lead,tail", SEGMENTS)
def test_segments(gpu_lib, lengths, n, k, act, lead, tail):
    host = segments_case(gen(sum(lengths) + n), lengths, n, k, lead, tail)
    qa, sa, seg, qb, sb = host
    rows = qa.shape[0]
    dev = [t.cuda() for t in host]
    zb, z = bf16_buffer(rows, 2 * n, 2 * n + 8)
    hb, h = bf16_buffer(rows, n, n + 8)
    cb, q = code_buffer(rows, n, n + 16)
    s = torch.full((rows, n // 128), NAN, device="cuda")
    gpu_lib.fp8bs_grouped_gemm_gated_ragged(*dev, act=ACTS[act], z=z, h=h, qh=q, sh=s)
    torch.cuda.synchronize()
    for e in range(len(lengths)):
        cut = slice(int(seg[e]), int(seg[e + 1]))
        if lengths[e]:
            z64, ez, h64, eh = gated64(qa[cut], sa[cut], qb[e], sb[e], act)
            check(z[cut], z64, ez, f"z of expert {e}")
            check(h[cut], h64, eh, f"h of expert {e}")
            check_codes(q[cut], s[cut], h64, eh, f"codes of expert {e}")
    out = torch.ones(rows, dtype=torch.bool)
    out[int(seg[0]):int(seg[-1])] = False
    assert z[out.cuda()].isnan().all() and h[out.cuda()].isnan().all() and s[out.cuda()].isnan().all()
    assert (q[out.cuda()] == 0x5A).all()
    assert untouched(zb, rows, 2 * n, NAN) and untouched(hb, rows, n, NAN) and untouched(cb, rows, n, 0x5A)
    only_h = torch.full((rows, n), NAN, dtype=torch.bfloat16, device="cuda")
    gpu_lib.fp8bs_grouped_gemm_gated_ragged(*dev, act=ACTS[act], h=only_h)
    for e in range(len(lengths)):
        cut = slice(int(seg[e]), int(seg[e + 1]))
        if lengths[e]:
            check(only_h[cut], *gated64(qa[cut], sa[cut], qb[e], sb[e], act)[2:], f"h alone of expert {e}")
    assert only_h[out.cuda()].isnan().all()
    if kernel(rows, n, k, False, len(lengths)) == kernel(rows, n, k, True, len(lengths)):
        assert torch.equal(only_h.view(torch.int16), h.contiguous().view(torch.int16))


def test_segments_that_hold_bad_offsets(gpu_lib):
    """Offsets outside the rows are clipped, a segment that runs backwards is empty: rows of one segment keep their results."""
    qa, sa, seg, qb, sb = segments_case(gen(3), [40, 30, 20, 10], 128, 256)
    bad = torch.tensor([-7, 40, 90, 60, 1000], dtype=torch.int32)     # rows 60 to 89 are in two segments
    h = torch.full((100, 128), NAN, dtype=torch.bfloat16, device="cuda")
    _, q, s = gpu_lib.fp8bs_grouped_gemm_gated_ragged(*(t.cuda() for t in (qa, sa, bad, qb, sb)), h=h, qh=None)
    torch.cuda.synchronize()
    for e, cut in ((0, slice(0, 40)), (3, slice(90, 100))):
        _, _, h64, eh = gated64(qa[cut], sa[cut], qb[e], sb[e], "silu")
        check(h[cut], h64, eh, f"expert {e}")


def test_no_rows(gpu_lib):
    n, k = 128, 256
    qb, sb = blocks(normal(gen(1), 3, 2 * n, k))
    h, q, s = gpu_lib.fp8bs_grouped_gemm_gated_ragged(
        torch.empty((0, k), dtype=torch.uint8, device="cuda"), torch.empty((0, k // 128), device="cuda"),
        torch.zeros(4, dtype=torch.int32, device="cuda"), qb.cuda(), sb.cuda(), qh=None)
    assert h.shape == (0, n) and q.shape == (0, n) and s.shape == (0, n // 128)
    got = gpu_lib.fp8bs_gated_backward(h, torch.empty((0, 2 * n), dtype=torch.bfloat16, device="cuda"), q=None, h=None)
    assert got[0].shape == (0, 2 * n) and got[1].shape == (0, 2 * n) and got[5].shape == (0, n)


def test_bindings_refusals(gpu_lib):
    g = gen(2)
    dev = [t.cuda() for t in operands(g, 4, 128, 256)]
    qa, sa, qb, sb = dev
    for bad in ((qa[:, :128], sa, qb, sb), (qa, sa[:2], qb, sb), (qa, sa, qb[:128], sb), (qa, sa, qb, sb[:1])):
        with pytest.raises((ValueError, gpu_lib.Fp8bsError)):
            gpu_lib.fp8bs_gemm_gated(*bad)
    with pytest.raises(gpu_lib.Fp8bsError):
        gpu_lib.fp8bs_gemm_gated(*dev, act=7)
    with pytest.raises(gpu_lib.Fp8bsError):
        gpu_lib.fp8bs_gemm_gated(*dev, h=False)
    with pytest.raises(ValueError):
        gpu_lib.fp8bs_gemm_gated(*dev, z=torch.empty((4, 128), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        gpu_lib.fp8bs_gemm_gated(*dev, sh=torch.empty((4, 1), device="cuda"))
    with pytest.raises(ValueError):
        gpu_lib.fp8bs_gemm_gated(*dev, qh=torch.empty((4, 64), dtype=torch.uint8, device="cuda"))
    long = [t.cuda() for t in operands(g, 4, 128, 7168)]
    assert gpu_lib.fp8bs_gemm_gated_workspace(4, 128, 7168) == 4 * 4 * 128
    with pytest.raises(gpu_lib.Fp8bsError):
        gpu_lib.fp8bs_gemm_gated(*long, qh=None, workspace=torch.empty(4, device="cuda"))
    dh, z = torch.zeros((128, 128), dtype=torch.bfloat16, device="cuda"), torch.zeros((128, 256), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        gpu_lib.fp8bs_gated_backward(dh, z[:, :128])
    with pytest.raises(gpu_lib.Fp8bsError):
        gpu_lib.fp8bs_gated_backward(dh, z, dz=False)
    with pytest.raises(gpu_lib.Fp8bsError):
        gpu_lib.fp8bs_gated_backward(dh[:100], z[:100], qt=None)
    with pytest.raises(gpu_lib.Fp8bsError):
        gpu_lib.fp8bs_gated_backward(dh, z, qt=None, row_end=torch.zeros(1, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        gpu_lib.fp8bs_gated_backward(dh, z, row_end=torch.zeros(2, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()


# ---- backward -----------------------------------------------------------------------------------


def backward_inputs(g, m, n, scale=1e-3):
    z = normal(g, m, 2 * n) * 1.5
    if m > 1:
        z[1, ::7] = 0.0
        z[1, 1::7] = -0.0
    if m > 3:
        z[2, ::5] = 40.0                          # saturated gates, both ways
        z[3, ::5] = -90.0
    return (normal(g, m, n) * scale).bfloat16(), z.bfloat16()


@pytest.mark.parametrize("m,n,act", [(1, 128, "silu"), (37, 1408, "silu"), (128, 128, "none"), (300, 256, "gelu_tanh"),
                                     (1000, 640, "relu"), (4100, 2048, "silu"), (9000, 1280, "gelu_tanh")])
def test_backward_rows(gpu_lib, m, n, act):
    dh, z = backward_inputs(gen(m + n), m, n)
    db, dhv = bf16_buffer(m, n, n + 8)
    zb, zv = bf16_buffer(m, 2 * n, 2 * n + 16)
    dhv.copy_(dh), zv.copy_(z)
    ob, dz = bf16_buffer(m, 2 * n, 2 * n + 24)
    hb, h = bf16_buffer(m, n, n + 40)
    cb, q = code_buffer(m, 2 * n, 2 * n + 48)
    s = torch.full((m, 2 * n // 128), NAN, device="cuda")
    out = gpu_lib.fp8bs_gated_backward(dhv, zv, act=ACTS[act], dz=dz, q=q, scales=s, h=h)
    torch.cuda.synchronize()
    assert out[0] is dz and out[1] is q and out[2] is s and out[5] is h and out[3] is None and out[6] is None
    w = backward64(dh, z, act)
    both = [torch.cat([w["dg"][i], w["du"][i]], 1) for i in (0, 1)]
    check(dz, *both, "dz")
    check(h, *w["h"], "h")
    check_codes(q, s, *both, "codes")
    assert untouched(ob, m, 2 * n, NAN) and untouched(hb, m, n, NAN) and untouched(cb, m, 2 * n, 0x5A)
    # in place, and one output at a time: the same bits
    bits = lambda t: t.contiguous().view(torch.int16)  # noqa: E731
    want_dz, want_h = bits(dz).clone(), bits(h).clone()
    only = gpu_lib.fp8bs_gated_backward(dhv, zv, act=ACTS[act], dz=False, q=None)
    assert torch.equal(only[1], q) and torch.equal(only[2], s) and only[0] is None
    gpu_lib.fp8bs_gated_backward(dhv, zv, act=ACTS[act], dz=zv, h=dhv)
    assert torch.equal(bits(zv), want_dz) and torch.equal(bits(dhv), want_h)
    torch.cuda.synchronize()


@pytest.mark.parametrize("n", [8, 40, 136, 1000])
def test_backward_of_widths_without_tiles(gpu_lib, n):
    dh, z = backward_inputs(gen(n), 67, n)
    got = gpu_lib.fp8bs_gated_backward(dh.cuda(), z.cuda(), act=3, h=None)
    w = backward64(dh, z, "silu")
    check(got[0], torch.cat([w["dg"][0], w["du"][0]], 1), torch.cat([w["dg"][1], w["du"][1]], 1), "dz")
    check(got[5], *w["h"], "h")


@pytest.mark.parametrize("m,n,act", [(128, 128, "silu"), (384, 256, "gelu_tanh"), (256, 640, "relu"), (1024, 1280, "none"),
                                     (4096, 2048, "silu"), (8192, 1408, "silu")])
def test_backward_both_orientations(gpu_lib, m, n, act):
    dh, z = backward_inputs(gen(m + n), m, n)
    w = backward64(dh, z, act)
    dhd, zd = dh.cuda(), z.cuda()
    dz, q, s, qt, st, h, qht, sht = gpu_lib.fp8bs_gated_backward(dhd, zd, act=ACTS[act], q=None, qt=None, h=None, qht=None)
    torch.cuda.synchronize()
    both = [torch.cat([w["dg"][i], w["du"][i]], 1) for i in (0, 1)]
    check_codes(q, s, *both, "codes along the columns")
    check_codes(qt, st, both[0].t().contiguous(), both[1].t().contiguous(), "codes along the rows")
    check_codes(qht, sht, w["h"][0].t().contiguous(), w["h"][1].t().contiguous(), "codes of h along the rows")
    # the kernel without transposed outputs makes the same bits of the others
    dz1, q1, s1, _, _, h1, _, _ = gpu_lib.fp8bs_gated_backward(dhd, zd, act=ACTS[act], q=None, h=None)
    for a, b in ((dz, dz1), (h, h1)):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    assert torch.equal(q, q1) and torch.equal(s, s1)
    # each transposed output alone, into wider buffers
    qb, qtv = code_buffer(2 * n, m, m + 16)
    st2 = torch.full((2 * n, m // 128), NAN, device="cuda")
    gpu_lib.fp8bs_gated_backward(dhd, zd, act=ACTS[act], dz=False, qt=qtv, scales_t=st2)
    assert torch.equal(qtv, qt) and torch.equal(st2, st) and untouched(qb, 2 * n, m, 0x5A)
    hb, qhv = code_buffer(n, m, m + 32)
    sh2 = torch.full((n, m // 128), NAN, device="cuda")
    gpu_lib.fp8bs_gated_backward(dhd, zd, act=ACTS[act], dz=False, qht=qhv, scales_ht=sh2)
    assert torch.equal(qhv, qht) and torch.equal(sh2, sht) and untouched(hb, n, m, 0x5A)
    # in place
    zz, dd = zd.clone(), dhd.clone()
    again = gpu_lib.fp8bs_gated_backward(dd, zz, act=ACTS[act], dz=zz, q=None, qt=None, h=dd, qht=None)
    for a, b in zip(again, (dz, q, s, qt, st, h, qht, sht)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("wide", ["z", "dz", "qt"])
def test_backward_of_the_largest_strides(gpu_lib, wide):
    """Rows 2^28 elements apart, less the alignment: offsets within a square pass 2^31, of a matrix 2^32."""
    m, n, stride = 128, 128, (1 << 28) - 16
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 100 GB of free memory")
    dh, z = backward_inputs(gen(28), m, n)
    dh, z = dh.cuda(), z.cuda()
    want = gpu_lib.fp8bs_gated_backward(dh, z, q=None, qt=None, h=None, qht=None)
    rows, cols, dtype = (2 * n, m, torch.uint8) if wide == "qt" else (m, 2 * n, torch.bfloat16)
    far = torch.empty(rows * stride, dtype=dtype, device="cuda").as_strided((rows, cols), (stride, 1))
    out = dict(dz=None, q=None, qt=None, h=None, qht=None)
    if wide == "z":
        z = far.copy_(z)
    elif wide == "dz":
        out["dz"] = far
    else:
        out.update(qt=far, scales_t=torch.empty(2 * n, 1, device="cuda"))
    got = gpu_lib.fp8bs_gated_backward(dh, z, **out)
    for a, b in zip(got, want):
        assert torch.equal(a.contiguous().view(torch.uint8), b.view(torch.uint8))
    del far, z, got, out
    torch.cuda.empty_cache()


@pytest.mark.parametrize("m,n,everything", [(8192, 2048, False), (16384, 2048, False), (16384, 2048, True)])
def test_large_backward_has_the_bits_of_its_parts(gpu_lib, m, n, everything):
    """Large calls pass through the caches in other ways (more than 128 MiB read and written, written, more than 256 MiB
    written): the same bits as calls on 2048 rows each."""
    g = gen(m)
    dh = (torch.randn(m, n, generator=g) * 1e-3).bfloat16().cuda()
    z = torch.randn(m, 2 * n, generator=g).bfloat16().cuda()
    extra = dict(h=None) if everything else dict(dz=False)
    whole = gpu_lib.fp8bs_gated_backward(dh, z, q=None, qt=None, qht=None, **extra)
    for r in range(0, m, 2048):
        part = gpu_lib.fp8bs_gated_backward(dh[r:r + 2048], z[r:r + 2048], q=None, qt=None, qht=None, **extra)
        for i, (a, b) in enumerate(zip(whole, part)):
            if b is None:
                assert a is None
                continue
            a = a[:, r // 128:r // 128 + 16] if i in (4, 7) else a[:, r:r + 2048] if i in (3, 6) else a[r:r + 2048]
            assert torch.equal(a.contiguous().view(torch.uint8), b.view(torch.uint8)), i


def test_backward_tiny_and_zero_groups(gpu_lib):
    """Gradients whose groups have subnormal scales, and groups of zeros, in both orientations."""
    m, n = 256, 256
    dh, z = backward_inputs(gen(9), m, n, scale=1.0)
    dh = dh.float()
    dh[:, :128] *= 2.0 ** -110
    dh[:64, 128:] = 0.0
    dh[64:70, 128:] *= 2.0 ** -133
    dh = dh.bfloat16()
    w = backward64(dh, z, "silu")
    got = gpu_lib.fp8bs_gated_backward(dh.cuda(), z.cuda(), dz=False, q=None, qt=None)
    both = [torch.cat([w["dg"][i], w["du"][i]], 1) for i in (0, 1)]
    check_codes(got[1], got[2], both[0], both[1] + 2.0 ** -148, "columns")
    check_codes(got[3], got[4], both[0].t().contiguous(), both[1].t().contiguous() + 2.0 ** -148, "rows")
    assert not (got[1][:64, 128:n] & 0x7F).any() and not got[2][:64, 1].any()


@pytest.mark.parametrize("end", [0, 1, 77, 100, 120])
def test_backward_row_end(gpu_lib, end):
    """Rows behind the last segment stay as they were."""
    m, n = 100, 384
    dh, z = backward_inputs(gen(end), m, n)
    dz = torch.full((m, 2 * n), NAN, dtype=torch.bfloat16, device="cuda")
    h = torch.full((m, n), NAN, dtype=torch.bfloat16, device="cuda")
    q = torch.full((m, 2 * n), 0x5A, dtype=torch.uint8, device="cuda")
    s = torch.full((m, 2 * n // 128), NAN, device="cuda")
    seg = torch.tensor([0, 3, end], dtype=torch.int32, device="cuda")
    gpu_lib.fp8bs_gated_backward(dh.cuda(), z.cuda(), dz=dz, q=q, scales=s, h=h, row_end=seg[-1:])
    live = min(end, m)
    w = backward64(dh, z, "silu")
    check(dz[:live], torch.cat([w["dg"][0], w["du"][0]], 1)[:live], torch.cat([w["dg"][1], w["du"][1]], 1)[:live], "dz")
    assert dz[live:].isnan().all() and h[live:].isnan().all() and s[live:].isnan().all() and (q[live:] == 0x5A).all()
    assert not dz[:live].isnan().any() and not h[:live].isnan().any() and not s[:live].isnan().any()


@pytest.mark.parametrize("act", sorted(ACTS))
def test_backward_against_differences(gpu_lib, act):
    """dz against central differences of the 64-bit h: the second difference bounds what they leave out."""
    m, n = 16, 64
    g = gen(len(act))
    z = (normal(g, m, 2 * n) * 1.5).bfloat16()
    z[:, :n] = torch.where(z[:, :n].abs() < 0.05, 0.5, z[:, :n].float()).bfloat16()   # away from relu's corner
    dh = torch.ones((m, n), dtype=torch.bfloat16)
    dz = gpu_lib.fp8bs_gated_backward(dh.cuda(), z.cuda(), act=ACTS[act])[0].cpu().double()
    from tests.linear_util import act64
    step = 2.0 ** -12
    h = lambda v: act64(v[:, :n], act) * v[:, n:]  # noqa: E731
    z64, up = z.double(), torch.zeros((m, 2 * n), dtype=torch.float64)
    for half in (slice(0, n), slice(n, 2 * n)):
        up.zero_()
        up[:, half] = step
        slope = (h(z64 + up) - h(z64 - up)) / (2 * step)
        # |act'''| < 4 for all of them; bf16 rounds to 2^-8
        allow = 2.0 ** -8 * slope.abs() + 4 * step ** 2 * (z64[:, n:].abs() + 1) + 2.0 ** -18 * (1 + z64[:, n:].abs())
        assert ((dz[:, half] - slope).abs() <= allow * 1.01).all()


# ---- as a program calls them --------------------------------------------------------------------


def test_streams_and_graphs(gpu_lib):
    """Calls on another stream, and captured ones: every replay gives the eager results, with eager work in between."""
    m, n, k = 260, 256, 512
    g = gen(11)
    dev = [t.cuda() for t in operands(g, m, n, k)]
    dh, z0 = (t.cuda() for t in backward_inputs(g, m, n))
    want = gpu_lib.fp8bs_gemm_gated(*dev, qh=None)
    want_b = gpu_lib.fp8bs_gated_backward(dh, z0, q=None, h=None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = gpu_lib.fp8bs_gemm_gated(*dev, qh=None, stream=side)
    got_b = gpu_lib.fp8bs_gated_backward(dh, z0, q=None, h=None, stream=side)
    side.synchronize()
    same = lambda a, b: all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b) if x is not None)  # noqa: E731
    assert same(want, got) and same(want_b, got_b)
    h, q, s = (torch.empty_like(t) for t in want)
    dz, bq, bs, bh = (torch.empty_like(want_b[i]) for i in (0, 1, 2, 5))
    ws = torch.empty(max(4, gpu_lib.fp8bs_gemm_gated_workspace(m, n, k) // 4), device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gpu_lib.fp8bs_gemm_gated(*dev, h=h, qh=q, sh=s, workspace=ws)
        gpu_lib.fp8bs_gated_backward(dh, z0, dz=dz, q=bq, scales=bs, h=bh)
    for _ in range(4):
        for t in (h, q, s, dz, bq, bs, bh):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert same(want, (h, q, s)) and same([want_b[i] for i in (0, 1, 2, 5)], (dz, bq, bs, bh))
        again = gpu_lib.fp8bs_gemm_gated(*dev, qh=None)
        assert same(want, again)


def test_two_calls_at_once(gpu_lib):
    """Two streams, a workspace each: neither disturbs the other."""
    n, k = 256, 1024
    cases = [[t.cuda() for t in operands(gen(20 + i), m, n, k)] for i, m in enumerate((40, 900))]
    want = [gpu_lib.fp8bs_gemm_gated(*c, qh=None) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(5):
        got = [gpu_lib.fp8bs_gemm_gated(*c, qh=None, stream=s) for c, s in zip(cases, streams)]
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


def test_code_values_feed_the_down_projection(gpu_lib):
    """The codes are what the quantizer's are to the next product: their product is near that of the bf16 h."""
    m, n, k, d = 200, 256, 512, 384
    g = gen(31)
    dev = [t.cuda() for t in operands(g, m, n, k)]
    wq, ws = (t.cuda() for t in blocks(normal(g, d, n) * 0.05))
    h, q, s = gpu_lib.fp8bs_gemm_gated(*dev, qh=None)
    y = gpu_lib.fp8bs_gemm(q, s, wq, ws)
    q2, s2 = gpu_lib.fp8bs_quantize_act_1x128(h)
    y2 = gpu_lib.fp8bs_gemm(q2, s2, wq, ws)
    value = q.view(E4M3).double() * s.double().repeat_interleave(128, 1)
    value2 = q2.view(E4M3).double() * s2.double().repeat_interleave(128, 1)
    # each is within half a step of h (2^-4), and h's own bf16 rounding
    assert ((value - value2).abs() <= 2.0 ** -3 * 1.01 * h.double().abs() + 2.0 ** -9 * (s + s2).double().repeat_interleave(128, 1)).all()
    w = wq.view(E4M3).double() * ws.double().repeat_interleave(128, 0).repeat_interleave(128, 1)
    off = (value - value2).abs() @ w.abs().t() + (2.0 ** -9 + 2.0 ** -7) * (value.abs() @ w.abs().t())
    assert ((y.double() - y2.double()).abs() <= off).all()
