"""Refusals of the linear-layer and ragged-expert entry points: host checks, no kernel is launched."""

import pytest
import torch

OK, ENULL, ESHAPE, EALIGN, EFLAG, ESCRATCH = 0, -1, -2, -3, -4, -6
P = 0x100000
BIG = 1 << 40


@pytest.fixture(scope="module")
def raw():
    from fp8_fine_grained_act_amd import lib

    return lib.raw


def call(fn, base, **change):
    """fn with the arguments of `base` (name -> value, in order), some changed."""
    assert set(change) <= set(base)
    return fn(*(change.get(k, v) for k, v in base.items()))


EPI = dict(qa=P, sa=P, qb=P, sb=P, m=4, n=128, k=128, b_layout=0, bias=P, act=3, res=P, ldr=128, z=P, ldz=128, c=P,
           ldc=128, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(qa=None), ENULL), (dict(sa=None), ENULL), (dict(qb=None), ENULL), (dict(sb=None), ENULL), (dict(c=None), ENULL),
    (dict(b_layout=2), EFLAG), (dict(act=4), EFLAG), (dict(act=-1), EFLAG),
    (dict(m=0), ESHAPE), (dict(m=-1), ESHAPE), (dict(n=100), ESHAPE), (dict(k=64), ESHAPE), (dict(k=0), ESHAPE),
    (dict(ldc=64), ESHAPE), (dict(ldr=120), ESHAPE), (dict(ldz=120), ESHAPE),
    (dict(qa=P + 8), EALIGN), (dict(c=P + 2), EALIGN), (dict(res=P + 8), EALIGN), (dict(z=P + 8), EALIGN),
    (dict(bias=P + 2), EALIGN), (dict(ldr=132), EALIGN), (dict(ldz=132), EALIGN), (dict(ldc=132), EALIGN),
    (dict(k=1 << 25), ESHAPE), (dict(b_layout=1, n=1 << 17, k=1 << 16, ldc=1 << 17, ldr=1 << 17, ldz=1 << 17), ESHAPE),
    (dict(m=BIG, n=1 << 21, ldc=1 << 21, ldr=1 << 21, ldz=1 << 21), ESHAPE),
])
def test_epilogue_refusals(raw, change, status):
    assert call(raw.fp8bs_gemm_epilogue, EPI, **change) == status


BWD = dict(dy=P, ldy=16, z=P, ldz=16, m=4, n=16, act=2, dz=P, lddz=16, dbias=P, accumulate=0, ws=None, ws_bytes=0,
           stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(dy=None), ENULL), (dict(z=None), ENULL), (dict(dz=None, dbias=None), ENULL),
    (dict(act=9), EFLAG), (dict(accumulate=2), EFLAG),
    (dict(m=0), ESHAPE), (dict(n=12), ESHAPE), (dict(n=0), ESHAPE), (dict(ldy=8), ESHAPE), (dict(ldz=8), ESHAPE),
    (dict(lddz=8), ESHAPE), (dict(m=BIG), ESHAPE),
    (dict(dy=P + 2), EALIGN), (dict(z=P + 8), EALIGN), (dict(dz=P + 8), EALIGN), (dict(ldy=20), EALIGN),
    (dict(ldz=20), EALIGN), (dict(lddz=20), EALIGN), (dict(dbias=P + 1), EALIGN), (dict(ws=P + 1), EALIGN),
    (dict(m=100000), ESCRATCH), (dict(m=100000, ws=P, ws_bytes=64), ESCRATCH),
])
def test_backward_refusals(raw, change, status):
    assert call(raw.fp8bs_epilogue_backward, BWD, **change) == status


def test_backward_workspace(raw):
    f = raw.fp8bs_epilogue_backward_workspace
    assert f(1, 8) == 0 and f(0, 8) == ESHAPE and f(4, 12) == ESHAPE and f(BIG, 8) == ESHAPE
    for m, n in ((16384, 4096), (100000, 8), (1 << 30, 8), (5000, 1 << 20)):
        b = f(m, n)
        assert b % (4 * n) == 0 and b // (4 * n) <= 65535 and (b > 0 or n >= 1 << 20), (m, n, b)


ROUTE = dict(ids=P, tokens=10, topk=4, experts=16, seg=P, slot=P, tok=P, cap=40, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(ids=None), ENULL), (dict(seg=None), ENULL), (dict(slot=None), ENULL), (dict(tok=None), ENULL),
    (dict(cap=39), ESHAPE), (dict(topk=0), ESHAPE), (dict(topk=65), ESHAPE), (dict(experts=513), ESHAPE),
    (dict(experts=0), ESHAPE), (dict(tokens=-1), ESHAPE), (dict(cap=1 << 31), ESHAPE),
    (dict(ids=P + 1), EALIGN), (dict(seg=P + 2), EALIGN),
])
def test_route_refusals(raw, change, status):
    assert call(raw.fp8bs_moe_route_ragged, ROUTE, **change) == status


GRP = dict(qa=P, sa=P, seg=P, experts=4, rows=100, qb=P, sb=P, n=128, k=128, b_layout=0, c=P, ldc=128, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(qa=None), ENULL), (dict(seg=None), ENULL), (dict(qb=None), ENULL), (dict(sb=None), ENULL), (dict(c=None), ENULL),
    (dict(b_layout=2), EFLAG), (dict(experts=0), ESHAPE), (dict(experts=65537), ESHAPE), (dict(rows=-1), ESHAPE),
    (dict(rows=1 << 30), ESHAPE), (dict(n=64), ESHAPE), (dict(k=192), ESHAPE), (dict(ldc=120), ESHAPE),
    (dict(k=1 << 25), ESHAPE), (dict(b_layout=1, n=1 << 17, k=1 << 16, ldc=1 << 17), ESHAPE),
    (dict(qa=P + 4), EALIGN), (dict(qb=P + 8), EALIGN), (dict(c=P + 8), EALIGN), (dict(seg=P + 2), EALIGN),
    (dict(ldc=132), EALIGN),
    (dict(rows=0), OK), (dict(rows=0, qa=None, sa=None, c=None), OK),
])
def test_grouped_refusals(raw, change, status):
    assert call(raw.fp8bs_grouped_gemm_ragged, GRP, **change) == status


WG = dict(dy=P, ldy=16, x=P, ldx=24, seg=P, experts=4, rows=100, m=16, n=24, c=P, accumulate=0, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(dy=None), ENULL), (dict(x=None), ENULL), (dict(seg=None), ENULL), (dict(c=None), ENULL),
    (dict(rows=0, c=None), ENULL), (dict(accumulate=2), EFLAG),
    (dict(experts=0), ESHAPE), (dict(experts=65537), ESHAPE), (dict(rows=-1), ESHAPE), (dict(rows=1 << 30), ESHAPE),
    (dict(m=12), ESHAPE), (dict(n=20), ESHAPE), (dict(m=0), ESHAPE), (dict(ldy=8), ESHAPE), (dict(ldx=16), ESHAPE),
    (dict(ldy=(1 << 24) + 8), ESHAPE), (dict(n=(1 << 21) + 8, ldx=(1 << 21) + 8), ESHAPE),
    (dict(experts=65536, m=1 << 16, n=1 << 16, ldy=1 << 16, ldx=1 << 16), ESHAPE),
    (dict(dy=P + 8), EALIGN), (dict(x=P + 2), EALIGN), (dict(c=P + 4), EALIGN), (dict(ldy=20), EALIGN),
    (dict(ldx=28), EALIGN), (dict(seg=P + 1), EALIGN),
])
def test_wgrad_refusals(raw, change, status):
    assert call(raw.fp8bs_grouped_wgrad_ragged, WG, **change) == status


def test_host_tensors_are_refused():
    from fp8_fine_grained_act_amd import lib

    u, f = torch.zeros((128, 128), dtype=torch.uint8), torch.ones((128, 1))
    b, seg = torch.zeros((128, 128), dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    for fn, args in ((lib.fp8bs_gemm_epilogue, (u, f, u, f)), (lib.fp8bs_epilogue_backward, (b, b)),
                     (lib.fp8bs_moe_route_ragged, (seg.view(1, 2), 4)),
                     (lib.fp8bs_grouped_gemm_ragged, (u, f, seg, u[None], f[None])),
                     (lib.fp8bs_grouped_wgrad_ragged, (b, b, seg))):
        with pytest.raises(TypeError):
            fn(*args)


@pytest.mark.gpu
def test_binding_refusals(gpu_lib):
    lib = gpu_lib
    d = dict(device="cuda")
    qa, sa = torch.zeros((5, 256), dtype=torch.uint8, **d), torch.ones((5, 2), **d)
    qb, sb = torch.zeros((128, 256), dtype=torch.uint8, **d), torch.ones((1, 2), **d)
    seg = torch.zeros(2, dtype=torch.int32, **d)
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, **d)  # noqa: E731
    bad = [
        lambda: lib.fp8bs_gemm_epilogue(qa, sa[:, :1].contiguous(), qb, sb),
        lambda: lib.fp8bs_gemm_epilogue(qa, sa, qb, sb, b_layout=1),
        lambda: lib.fp8bs_gemm_epilogue(qa, sa, qb, sb, bias=torch.zeros(64, **d)),
        lambda: lib.fp8bs_gemm_epilogue(qa, sa, qb, sb, residual=bf(4, 128)),
        lambda: lib.fp8bs_gemm_epilogue(qa, sa, qb, sb, c=bf(128, 5).t()),
        lambda: lib.fp8bs_epilogue_backward(bf(4, 16), None, act=3),
        lambda: lib.fp8bs_epilogue_backward(bf(4, 16), bf(4, 24), act=3),
        lambda: lib.fp8bs_epilogue_backward(bf(4, 16), bf(4, 16), accumulate=1),
        lambda: lib.fp8bs_grouped_gemm_ragged(qa, sa, seg, qb, sb),
        lambda: lib.fp8bs_grouped_gemm_ragged(qa, sa, torch.zeros(3, dtype=torch.int32, **d), qb[None], sb[None]),
        lambda: lib.fp8bs_grouped_wgrad_ragged(bf(4, 16), bf(5, 16), seg),
        lambda: lib.fp8bs_grouped_wgrad_ragged(bf(4, 16), bf(4, 16), seg, c=torch.zeros((2, 16, 16), **d)),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was not refused")
    for f in (lambda: lib.fp8bs_gemm_epilogue(qa, sa, qb, sb, act=7),
              lambda: lib.fp8bs_epilogue_backward(bf(5000, 512), bf(5000, 512), act=3, workspace=torch.zeros(4, **d)),
              lambda: lib.fp8bs_grouped_wgrad_ragged(bf(4, 12), bf(4, 16), seg)):
        with pytest.raises(lib.Fp8bsError):
            f()
    torch.cuda.synchronize()                                      # the refusals left the device usable
