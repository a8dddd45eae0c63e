"""The linear layer's epilogue and its backward pass on the GPU against 64-bit plain forms.

The bounds are derived in linear_util.
"""

import pytest
import torch

from tests.linear_util import (ACTS, SLOPE, act64, argument, blocks, check, gen, normal, product64, row_tiles,
                               slope64)

pytestmark = pytest.mark.gpu


def operands(g, m, n, k, b_layout):
    qa, sa = row_tiles(normal(g, m, k) * (1 + 20 * (torch.rand(k, generator=g) < 0.01)))
    qb, sb = blocks(normal(g, *((n, k) if b_layout == 0 else (k, n))) * 0.05)
    return qa, sa, qb, sb


def expected(ops, b_layout, bias, act, residual):
    z, e = product64(*ops, b_layout)
    if bias is not None:
        z = z + bias.double()
        e = e + 2.0 ** -24 * (z.abs() + e)
    y = act64(z, act)
    ey = (SLOPE if act != "none" else 1.0) * e + (argument(z, act) + 4) * 2.0 ** -24 * z.abs()
    if residual is not None:
        y = y + residual.double()
        ey = ey + 2.0 ** -24 * (y.abs() + ey)
    return z, e, y, ey


# one row to several tiles, around every tile edge; few and many columns; one to many blocks
SIZES = [(1, 128, 128), (2, 256, 384), (15, 384, 256), (16, 128, 1024), (17, 640, 512), (33, 256, 2048),
         (63, 1536, 128), (64, 128, 7168), (65, 512, 640), (127, 256, 256), (200, 1152, 384), (257, 384, 1024)]


@pytest.mark.parametrize("b_layout", [0, 1])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_epilogue_matches_64_bits(gpu_lib, m, n, k, b_layout):
    g = gen(m * 7 + n + k + b_layout)
    ops = operands(g, m, n, k, b_layout)
    dev = [t.cuda() for t in ops]
    for act, has_bias, has_res, has_z in (("none", 0, 0, 0), ("silu", 1, 0, 0), ("gelu_tanh", 1, 1, 1),
                                          ("relu", 0, 1, 0), ("none", 1, 1, 1)):
        bias = normal(g, n) if has_bias else None
        res = normal(g, m, n).bfloat16() if has_res else None
        z = torch.full((m, n), float("nan"), dtype=torch.bfloat16, device="cuda") if has_z else None
        c = gpu_lib.fp8bs_gemm_epilogue(*dev, b_layout=b_layout, bias=None if bias is None else bias.cuda(),
                                        act=ACTS[act], residual=None if res is None else res.cuda(), z=z)
        torch.cuda.synchronize()
        z64, ez, y64, ey = expected(ops, b_layout, bias, act, res)
        check(c, y64, ey, f"{m}x{n}x{k} layout {b_layout} {act}")
        if has_z:
            check(z, z64, ez, f"{m}x{n}x{k} layout {b_layout} z")


def test_no_epilogue_equals_the_plain_product(gpu_lib):
    """Without bias, act and residual the call computes fp8bs_gemm (same bound, both layouts, larger shapes)."""
    for m, n, k, b_layout in ((300, 1536, 7168, 0), (4096, 640, 7168, 0), (2048, 2048, 512, 0), (1037, 7168, 1536, 1),
                              (4096, 512, 8192, 1)):
        g = gen(m + n)
        ops = operands(g, m, n, k, b_layout)
        dev = [t.cuda() for t in ops]
        c = gpu_lib.fp8bs_gemm_epilogue(*dev, b_layout=b_layout)
        r = gpu_lib.fp8bs_gemm(*dev, b_layout=b_layout)
        a = dev[0].view(torch.float8_e4m3fn).float() * dev[1].repeat_interleave(128, 1)
        b = dev[2].view(torch.float8_e4m3fn).float() * dev[3].repeat_interleave(128, 0).repeat_interleave(128, 1)
        mag = (a.abs() @ (b.abs().t() if b_layout == 0 else b.abs())).double().cpu()
        e = (2.0 ** -10 + (k // 128 + 2) * 2.0 ** -24) * mag
        # both carry the product's error and one bf16 rounding
        check(c, r.double().cpu(), 2 * e + 2.0 ** -8 * r.double().cpu().abs(), f"{m}x{n}x{k}")


@pytest.mark.parametrize("m", [3, 70, 300])
@pytest.mark.parametrize("b_layout", [0, 1])
def test_epilogue_strides_residual_in_place_and_untouched_surroundings(gpu_lib, m, b_layout):
    n, k = 256, 256
    g = gen(5 + m)
    ops = operands(g, m, n, k, b_layout)
    dev = [t.cuda() for t in ops]
    bias, res = normal(g, n), normal(g, m, n).bfloat16()
    big = torch.full((m + 2, n + 24), 7.0, dtype=torch.bfloat16, device="cuda")
    zbig = torch.full((m + 2, n + 8), 5.0, dtype=torch.bfloat16, device="cuda")
    c, z = big[1:m + 1, 8:8 + n], zbig[1:m + 1, :n]
    c.copy_(res)
    out = gpu_lib.fp8bs_gemm_epilogue(*dev, b_layout=b_layout, bias=bias.cuda(), act=ACTS["gelu_tanh"], residual=c, z=z,
                                      c=c)
    torch.cuda.synchronize()
    assert out.data_ptr() == c.data_ptr()
    z64, ez, y64, ey = expected(ops, b_layout, bias, "gelu_tanh", res)
    check(c, y64, ey, "residual in place")
    check(z, z64, ez, "strided z")
    keep = torch.ones_like(big, dtype=torch.bool)
    keep[1:m + 1, 8:8 + n] = False
    assert (big[keep] == 7.0).all()
    keep = torch.ones_like(zbig, dtype=torch.bool)
    keep[1:m + 1, :n] = False
    assert (zbig[keep] == 5.0).all()


@pytest.mark.parametrize("act", ["gelu_tanh", "silu", "relu"])
def test_epilogue_of_large_values(gpu_lib, act):
    """Pre-activations from 1e-30 to 1e30: sigma saturates, nothing overflows to NaN."""
    m, n, k = 4, 128, 128
    qa = torch.zeros((m, k), dtype=torch.uint8)
    qa[:, 0] = 0x38                                              # 1.0
    sa = torch.ones((m, 1))
    qb = torch.zeros((n, k), dtype=torch.uint8)
    sb = torch.ones((1, 1))
    e = torch.linspace(-30, 30, n)
    bias = (10.0 ** e) * torch.where(torch.arange(n) % 2 == 0, 1.0, -1.0)
    c = gpu_lib.fp8bs_gemm_epilogue(qa.cuda(), sa.cuda(), qb.cuda(), sb.cuda(), bias=bias.cuda(), act=ACTS[act])
    torch.cuda.synchronize()
    z = bias.double().expand(m, n)
    y = z.clamp(min=0) if act == "relu" else act64(z, act)
    check(c, y, (argument(z, act) + 4) * 2.0 ** -24 * z.abs() * (z.abs() < 104), act)


def test_epilogue_on_another_stream_and_captured(gpu_lib):
    g = gen(11)
    for m in (4, 96, 300):
        ops = operands(g, m, 512, 1024, 0)
        dev = [t.cuda() for t in ops]
        bias = normal(g, 512).cuda()
        c = torch.empty((m, 512), dtype=torch.bfloat16, device="cuda")
        want = gpu_lib.fp8bs_gemm_epilogue(*dev, bias=bias, act=ACTS["silu"])
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        gpu_lib.fp8bs_gemm_epilogue(*dev, bias=bias, act=ACTS["silu"], c=c, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(c.view(torch.int16), want.view(torch.int16))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            gpu_lib.fp8bs_gemm_epilogue(*dev, bias=bias, act=ACTS["silu"], c=c)
        for _ in range(3):
            dev[0].copy_(dev[0].flip(0))
            want = gpu_lib.fp8bs_gemm_epilogue(*dev, bias=bias, act=ACTS["silu"])
            c.fill_(float("nan"))
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(c.view(torch.int16), want.view(torch.int16))


# ---- backward -----------------------------------------------------------------------------------

BWD = [(1, 8), (1, 1024), (2, 16), (3, 520), (37, 1536), (64, 512), (65, 8), (129, 2048), (1000, 72), (5000, 512),
       (700, 4096)]


def bwd64(dy, z, act):
    """(dz, its error, dbias, its error): the slope's error as act's (see linear_util), relative to 1 + |v|."""
    zd, d = z.double(), dy.double()
    s = slope64(zd, act)
    e = d.abs() * (2 * argument(zd, act) + 8) * 2.0 ** -24 * (1 + zd.abs().clamp(max=104) * (act != "none"))
    dz = d * s
    m = dy.shape[0]
    # the column sum: at most m FP32 additions of partial sums bounded by sum |dz|
    return dz, e, dz.sum(0), e.sum(0) + m * 2.0 ** -24 * (dz.abs() + e).sum(0)


@pytest.mark.parametrize("act", sorted(ACTS))
@pytest.mark.parametrize("m,n", BWD)
def test_backward_matches_64_bits(gpu_lib, m, n, act):
    g = gen(m + n)
    dy, z = (normal(g, m, n) * 1e-2).bfloat16(), (normal(g, m, n) * 2).bfloat16()
    dz, db = gpu_lib.fp8bs_epilogue_backward(dy.cuda(), z.cuda(), act=ACTS[act])
    torch.cuda.synchronize()
    dz64, e, db64, eb = bwd64(dy, z, act)
    check(dz, dz64, e, f"{act} dz")
    check(db, db64, eb, f"{act} dbias", bf16=False)


def test_backward_modes(gpu_lib):
    """In place, strided, accumulate, one result only, given workspace, z absent."""
    g = gen(3)
    for m, n in ((50, 520), (900, 1024)):
        dy, z = normal(g, m, n).bfloat16(), normal(g, m, n).bfloat16()
        dz64, e, db64, eb = bwd64(dy, z, "silu")
        big = torch.full((m + 1, n + 16), 3.0, dtype=torch.bfloat16, device="cuda")
        d = big[:m, 8:8 + n]
        d.copy_(dy)
        base = normal(g, n)
        db = base.cuda()
        need = gpu_lib.fp8bs_epilogue_backward_workspace(m, n)
        ws = torch.empty(need // 4 + 5, device="cuda")
        out, db2 = gpu_lib.fp8bs_epilogue_backward(d, z.cuda(), act=ACTS["silu"], dz=d, dbias=db, accumulate=1,
                                                   workspace=ws)
        torch.cuda.synchronize()
        assert out.data_ptr() == d.data_ptr() and db2.data_ptr() == db.data_ptr()
        check(d, dz64, e, "in place")
        tot = base.double() + db64
        check(db, tot, eb + 2.0 ** -24 * (tot.abs() + eb), "accumulated", bf16=False)
        assert (big[m:] == 3.0).all() and (big[:, :8] == 3.0).all() and (big[:, 8 + n:] == 3.0).all()
        only, none = gpu_lib.fp8bs_epilogue_backward(dy.cuda(), z.cuda(), act=ACTS["silu"], dbias=False)
        assert none is None and torch.equal(only.view(torch.int16), d.contiguous().view(torch.int16))
        none, only = gpu_lib.fp8bs_epilogue_backward(dy.cuda(), z.cuda(), act=ACTS["silu"], dz=False)
        assert none is None
        check(only, db64, eb, "dbias only", bf16=False)
        dz, db = gpu_lib.fp8bs_epilogue_backward(dy.cuda(), None)
        assert torch.equal(dz.cpu().view(torch.int16), dy.view(torch.int16))
        check(db, dy.double().sum(0), m * 2.0 ** -24 * dy.double().abs().sum(0), "no act", bf16=False)


@pytest.mark.parametrize("act", ["gelu_tanh", "silu"])
def test_backward_of_large_values(gpu_lib, act):
    mags = torch.tensor([0.0, 1e-30, 1e-3, 0.5, 3.0, 12.0, 15.9, 16.1, 80.0, 90.0, 1e4, 1e15, 1e25, 3e38])
    z = torch.cat([mags, -mags, mags, -mags[:14]])[:56].bfloat16().reshape(1, 56)
    dy = torch.ones_like(z)
    dz, _ = gpu_lib.fp8bs_epilogue_backward(dy.cuda(), z.cuda(), act=ACTS[act])
    torch.cuda.synchronize()
    zd = z.double()
    want = torch.where(zd.abs() < 60, slope64(zd.clamp(-60, 60), act), (zd > 0).double())
    e = (2 * argument(zd, act) + 8) * 2.0 ** -24 * (1 + zd.abs().clamp(max=104))
    check(dz, want, e, act)


def test_backward_against_differences_of_the_forward(gpu_lib):
    """dz is the derivative of the forward's act, bias and residual: central differences of a 64-bit loss
    sum(y * w) taken through the forward's own formula at the kernel's z."""
    g = gen(9)
    z = (normal(g, 6, 64) * 2).bfloat16()
    w = normal(g, 6, 64).bfloat16()
    for act in ("gelu_tanh", "silu"):
        dz, db = gpu_lib.fp8bs_epilogue_backward(w.cuda(), z.cuda(), act=ACTS[act])
        h = 1e-5
        zd = z.double()
        diff = (act64(zd + h, act) - act64(zd - h, act)) / (2 * h) * w.double()
        # central differences: h^2/6 of the third derivative (below 3) and 2^-52 |act| / h of cancellation
        e = w.double().abs() * (3 * h * h + 2.0 ** -52 * zd.abs() / h * 4 + 3e-5)
        check(dz, diff, e, act)
        check(db, diff.sum(0), e.sum(0) + 6 * 2.0 ** -24 * diff.abs().sum(0), act, bf16=False)


def test_backward_graph_replays(gpu_lib):
    g = gen(13)
    m, n = 3000, 1024
    dy, z = normal(g, m, n).bfloat16().cuda(), normal(g, m, n).bfloat16().cuda()
    dz, db = torch.empty_like(dy), torch.empty(n, device="cuda")
    ws = torch.empty(gpu_lib.fp8bs_epilogue_backward_workspace(m, n) // 4, device="cuda")
    gpu_lib.fp8bs_epilogue_backward(dy, z, act=3, dz=dz, dbias=db, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gpu_lib.fp8bs_epilogue_backward(dy, z, act=3, dz=dz, dbias=db, workspace=ws)
    for i in range(3):
        z.copy_(z.roll(i + 1, 0))
        dz2, db2 = gpu_lib.fp8bs_epilogue_backward(dy, z, act=3)
        dz.fill_(0)
        db.fill_(0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(dz.view(torch.int16), dz2.view(torch.int16)) and torch.equal(db, db2)


@pytest.mark.parametrize("b_layout", [0, 1])
@pytest.mark.parametrize("m,n,k", [(500, 1536, 1024), (1000, 1536, 512), (1100, 2048, 256), (2048, 2048, 512),
                                   (1037, 7168, 256), (4096, 4096, 256), (4096, 1536, 384), (3000, 8192, 128),
                                   (16, 8192, 256), (40, 7168, 384), (250, 2048, 640)])
def test_epilogue_on_every_tile_shape(gpu_lib, m, n, k, b_layout):
    """Products over one round of the chip and more: every tile shape, persistent workgroups, ragged last tiles."""
    g = gen(m + n + k)
    ops = operands(g, m, n, k, b_layout)
    bias, res = normal(g, n), normal(g, m, n).bfloat16()
    dev = [t.cuda() for t in ops]
    z = torch.empty((m, n), dtype=torch.bfloat16, device="cuda")
    c = gpu_lib.fp8bs_gemm_epilogue(*dev, b_layout=b_layout, bias=bias.cuda(), act=ACTS["gelu_tanh"], residual=res.cuda(),
                                    z=z)
    torch.cuda.synchronize()
    z64, ez = product64(*dev, b_layout)
    z64, ez = z64.cpu(), ez.cpu()
    z64 = z64 + bias.double()
    ez = ez + 2.0 ** -24 * (z64.abs() + ez)
    y = act64(z64, "gelu_tanh") + res.double()
    ey = SLOPE * ez + (argument(z64, "gelu_tanh") + 4) * 2.0 ** -24 * z64.abs()
    check(z, z64, ez, "z")
    check(c, y, ey + 2.0 ** -24 * (y.abs() + ey), "c")


def test_backward_calls_at_once_on_two_streams(gpu_lib):
    """Each call's outputs and workspace are its own, also where the call makes them."""
    g = gen(17)
    m, n = 9000, 1024
    dy = [normal(g, m, n).bfloat16().cuda() for _ in range(2)]
    z = normal(g, m, n).bfloat16().cuda()
    want = [gpu_lib.fp8bs_epilogue_backward(d, z, act=ACTS["gelu_tanh"]) for d in dy]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in dy]
    got = [[], []]
    for _ in range(4):
        for i, s in enumerate(streams):
            got[i].append(gpu_lib.fp8bs_epilogue_backward(dy[i], z, act=ACTS["gelu_tanh"], stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        for dz, db in got[i]:
            assert torch.equal(dz.view(torch.int16), want[i][0].view(torch.int16)) and torch.equal(db, want[i][1])


def test_not_a_number_stays_one(gpu_lib):
    """NaN and infinities of a row reach that row's outputs and its columns' sums, and nothing else."""
    m, n = 70, 1024
    g = gen(23)
    dy, z = normal(g, m, n).bfloat16(), normal(g, m, n).bfloat16()
    clean = gpu_lib.fp8bs_epilogue_backward(dy.cuda(), z.cuda(), act=ACTS["silu"])
    nan = torch.tensor([0x7FFF], dtype=torch.int16).view(torch.bfloat16)       # the payload that an integer rounding loses
    dy[3, 5], dy[4, 6], dy[5, 7] = nan[0], float("inf"), float("-inf")
    dz, db = gpu_lib.fp8bs_epilogue_backward(dy.cuda(), z.cuda(), act=ACTS["silu"])
    torch.cuda.synchronize()
    assert torch.isnan(dz[3, 5]) and torch.isnan(db[5]) and torch.isinf(dz[4, 6]) and torch.isinf(db[6]) and torch.isinf(db[7])
    keep = torch.ones((m, n), dtype=torch.bool)
    keep[3, 5] = keep[4, 6] = keep[5, 7] = False
    assert torch.equal(dz.cpu()[keep], clean[0].cpu()[keep])
    cols = torch.ones(n, dtype=torch.bool)
    cols[5:8] = False
    assert torch.equal(db.cpu()[cols], clean[1].cpu()[cols])
    # the forward: a NaN bias column and a NaN residual value
    qa, sa = row_tiles(normal(g, m, 256))
    qb, sb = blocks(normal(g, n, 256) * 0.05)
    dev = [t.cuda() for t in (qa, sa, qb, sb)]
    bias, res = torch.zeros(n), torch.zeros((m, n), dtype=torch.bfloat16)
    y0 = gpu_lib.fp8bs_gemm_epilogue(*dev, bias=bias.cuda(), act=ACTS["gelu_tanh"], residual=res.cuda()).cpu()
    bias[9], res[2, 11] = float("nan"), nan[0]
    y = gpu_lib.fp8bs_gemm_epilogue(*dev, bias=bias.cuda(), act=ACTS["gelu_tanh"], residual=res.cuda()).cpu()
    assert torch.isnan(y[:, 9]).all() and torch.isnan(y[2, 11])
    keep = torch.ones((m, n), dtype=torch.bool)
    keep[:, 9] = keep[2, 11] = False
    assert torch.equal(y[keep], y0[keep])
    # a NaN pre-activation: no activation hides it, and the smooth slopes keep it
    for act in ("relu", "gelu_tanh", "silu"):
        y = gpu_lib.fp8bs_gemm_epilogue(*dev, bias=bias.cuda(), act=ACTS[act]).cpu()
        assert torch.isnan(y[:, 9]).all() and int(torch.isnan(y).sum()) == m, act
    for act in ("gelu_tanh", "silu"):
        dz, _ = gpu_lib.fp8bs_epilogue_backward(torch.ones_like(z).cuda(), torch.full_like(z, float("nan")).cuda(), act=ACTS[act])
        assert torch.isnan(dz).all(), act


@pytest.mark.parametrize("m,n", [(511, 200), (512, 1032), (513, 64), (300, 4096), (9, 65544)])
def test_backward_around_the_row_limit_of_one_launch(gpu_lib, m, n):
    g = gen(m)
    dy, z = (normal(g, m, n) * 1e-2).bfloat16(), (normal(g, m, n) * 2).bfloat16()
    base = normal(g, n)
    db = base.cuda()
    assert (gpu_lib.fp8bs_epilogue_backward_workspace(m, n) == 0) == (m <= 512)
    dz, _ = gpu_lib.fp8bs_epilogue_backward(dy.cuda(), z.cuda(), act=ACTS["gelu_tanh"], dbias=db, accumulate=1)
    torch.cuda.synchronize()
    dz64, e, db64, eb = bwd64(dy, z, "gelu_tanh")
    check(dz, dz64, e, "dz")
    tot = base.double() + db64
    check(db, tot, eb + 2.0 ** -24 * (tot.abs() + eb), "dbias", bf16=False)
