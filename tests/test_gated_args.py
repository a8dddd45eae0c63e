"""Refusals of the gated block's and the optimizer's entry points: host checks, no kernel is launched."""

import ctypes

import pytest
import torch

OK, ENULL, ESHAPE, EALIGN, EFLAG, ESCRATCH = 0, -1, -2, -3, -4, -6
P = 0x100000
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    from fp8_fine_grained_act_amd import lib

    return lib


def call(fn, base, **change):
    """fn with the arguments of `base` (name -> value, in order), some changed."""
    assert set(change) <= set(base)
    return fn(*(change.get(k, v) for k, v in base.items()))


OUTS = dict(act=3, z=P, ldz=256, h=P, ldh=128, qh=P, ldqh=128, sh=P, ws=P, ws_bytes=0, stream=None)
FWD = dict(qa=P, sa=P, qb=P, sb=P, m=4, n=128, k=128, **OUTS)
RAG = dict(qa=P, sa=P, seg=P, experts=2, rows=4, qb=P, sb=P, n=128, k=128, **OUTS)
SHARED = [
    (dict(qa=None), ENULL), (dict(sa=None), ENULL), (dict(qb=None), ENULL), (dict(sb=None), ENULL),
    (dict(h=None, qh=None, sh=None), ENULL), (dict(qh=None), ENULL), (dict(sh=None), ENULL),
    (dict(act=4), EFLAG), (dict(act=-1), EFLAG),
    (dict(n=100), ESHAPE), (dict(n=0), ESHAPE), (dict(k=64), ESHAPE), (dict(k=0), ESHAPE), (dict(k=-128), ESHAPE),
    (dict(ldz=248), ESHAPE), (dict(ldh=120), ESHAPE), (dict(ldqh=112), ESHAPE), (dict(k=1 << 24), ESHAPE),
    (dict(k=1 << 56), ESHAPE), (dict(k=(1 << 63) - 128), ESHAPE), (dict(n=1 << 61, ldz=1 << 62, ldh=1 << 61, ldqh=1 << 61), ESHAPE),
    (dict(n=1 << 16, k=1 << 15, ldz=1 << 17, ldh=1 << 16, ldqh=1 << 16), ESHAPE),
    (dict(qa=P + 8), EALIGN), (dict(qb=P + 8), EALIGN), (dict(sa=P + 2), EALIGN), (dict(sb=P + 2), EALIGN),
    (dict(z=P + 8), EALIGN), (dict(h=P + 8), EALIGN), (dict(qh=P + 8), EALIGN), (dict(sh=P + 2), EALIGN),
    (dict(ldz=260), EALIGN), (dict(ldh=132), EALIGN), (dict(ldqh=136), EALIGN), (dict(ws=P + 4), EALIGN),
]


@pytest.mark.parametrize("change,status", SHARED + [(dict(m=0), ESHAPE), (dict(m=-1), ESHAPE), (dict(m=BIG), ESHAPE)])
def test_gated_refusals(lib, change, status):
    assert call(lib.raw.fp8bs_gemm_gated, FWD, **change) == status


def test_gated_workspace_refusals(lib):
    """Few rows over a long contraction make their codes through the workspace: none, or one byte too small."""
    need = lib.raw.fp8bs_gemm_gated_workspace(4, 128, 7168)
    assert need == lib.raw.fp8bs_grouped_gemm_gated_ragged_workspace(2, 4, 128, 7168) == 4 * 4 * 128
    for change in (dict(ws=None, ws_bytes=need), dict(ws_bytes=need - 1), dict(ws_bytes=0)):
        assert call(lib.raw.fp8bs_gemm_gated, FWD, k=7168, **change) == ESCRATCH
        assert call(lib.raw.fp8bs_grouped_gemm_gated_ragged, RAG, k=7168, **change) == ESCRATCH


@pytest.mark.parametrize("change,status", SHARED + [
    (dict(seg=None), ENULL), (dict(seg=P + 2), EALIGN), (dict(experts=0), ESHAPE), (dict(experts=65537), ESHAPE),
    (dict(rows=-1), ESHAPE), (dict(rows=1 << 30), ESHAPE)])
def test_gated_ragged_refusals(lib, change, status):
    assert call(lib.raw.fp8bs_grouped_gemm_gated_ragged, RAG, **change) == status


def test_gated_ragged_without_rows(lib):
    assert call(lib.raw.fp8bs_grouped_gemm_gated_ragged, RAG, rows=0, qa=None, sa=None, z=None, h=None, qh=None, sh=None,
                ws=None) == OK


def test_gated_workspaces(lib):
    f, g = lib.raw.fp8bs_gemm_gated_workspace, lib.raw.fp8bs_grouped_gemm_gated_ragged_workspace
    assert 0 <= f(4, 128, 128) <= 4 * 4 * 128
    assert 0 <= f(1000, 2048, 7168) <= 4 * 1000 * 2048
    assert g(4, 0, 128, 128) == 0
    assert 0 <= g(4, 100, 256, 128) <= 4 * 100 * 256
    for args in ((0, 128, 128), (4, 100, 128), (4, 128, 0), (4, 0, 128), (BIG, 128, 128), (-1, 128, 128)):
        assert f(*args) == ESHAPE
    for args in ((0, 4, 128, 128), (65537, 4, 128, 128), (4, -1, 128, 128), (4, 1 << 30, 128, 128), (4, 4, 100, 128)):
        assert g(*args) == ESHAPE
    with pytest.raises(lib.Fp8bsError):
        lib.fp8bs_gemm_gated_workspace(4, 100, 128)


BWD = dict(dh=P, lddh=128, z=P, ldz=256, m=128, n=128, act=3, dz=P, lddz=256, q=P, ldq=256, s=P, qt=P, ldqt=128, st=P, h=P,
           ldh=128, qht=P, ldqht=128, sht=P, row_end=None, stream=None)
NONE = dict(dz=None, q=None, s=None, qt=None, st=None, h=None, qht=None, sht=None)


@pytest.mark.parametrize("change,status", [
    (dict(dh=None), ENULL), (dict(z=None), ENULL), (dict(s=None), ENULL), (dict(q=None), ENULL), (dict(st=None), ENULL),
    (dict(qt=None), ENULL), (dict(sht=None), ENULL), (dict(qht=None), ENULL), (NONE, ENULL),
    (dict(act=9), EFLAG), (dict(act=-1), EFLAG),
    (dict(m=-128), ESHAPE), (dict(n=0), ESHAPE), (dict(n=136, lddh=136, ldz=272, lddz=272, ldq=272, ldh=136), ESHAPE),
    (dict(m=100), ESHAPE), (dict(row_end=P), ESHAPE), (dict(m=1 << 23, ldqt=1 << 23, ldqht=1 << 23), ESHAPE),
    (dict(NONE, dz=P, n=12, lddh=16, ldz=24, lddz=24), ESHAPE), (dict(NONE, dz=P, m=BIG), ESHAPE),
    (dict(lddh=120), ESHAPE), (dict(ldz=248), ESHAPE), (dict(lddz=248), ESHAPE), (dict(ldq=240), ESHAPE),
    (dict(ldqt=112), ESHAPE), (dict(ldh=120), ESHAPE), (dict(ldqht=112), ESHAPE),
    (dict(dh=P + 8), EALIGN), (dict(z=P + 2), EALIGN), (dict(dz=P + 8), EALIGN), (dict(q=P + 8), EALIGN),
    (dict(qt=P + 8), EALIGN), (dict(h=P + 8), EALIGN), (dict(qht=P + 8), EALIGN), (dict(s=P + 2), EALIGN),
    (dict(st=P + 1), EALIGN), (dict(sht=P + 2), EALIGN), (dict(lddh=132), EALIGN), (dict(ldz=260), EALIGN),
    (dict(lddz=260), EALIGN), (dict(ldq=264), EALIGN), (dict(ldqt=136), EALIGN), (dict(ldh=132), EALIGN),
    (dict(ldqht=136), EALIGN), (dict(NONE, dz=P, row_end=P + 2), EALIGN),
])
def test_gated_backward_refusals(lib, change, status):
    assert call(lib.raw.fp8bs_gated_backward, BWD, **change) == status


def test_gated_backward_without_rows(lib):
    assert call(lib.raw.fp8bs_gated_backward, BWD, m=0) == OK
    assert call(lib.raw.fp8bs_gated_backward, BWD, **dict(NONE, m=0, dh=None, z=None)) == OK


@pytest.mark.parametrize("stride", ["lddh", "ldz", "lddz", "ldq", "ldqt", "ldh", "ldqht"])
def test_gated_backward_stride_limit_of_transposed_outputs(lib, stride):
    assert call(lib.raw.fp8bs_gated_backward, BWD, **{stride: 1 << 28}) == ESHAPE
    assert call(lib.raw.fp8bs_gated_backward, BWD, **{stride: (1 << 28) - 16, "m": 0}) == OK
    without = dict(NONE, dz=P, q=P, s=P, h=P, m=0)
    assert call(lib.raw.fp8bs_gated_backward, BWD, **{**without, stride: 1 << 28}) == OK
    alone = dict(NONE, qt=P, st=P, m=0)          # strides of outputs that are left out do not count
    assert call(lib.raw.fp8bs_gated_backward, BWD, **{**alone, stride: 1 << 28}) == \
        (ESHAPE if stride in ("lddh", "ldz", "ldqt") else OK)
    assert call(lib.raw.fp8bs_gated_backward, BWD, m=0, act=9) == EFLAG


STEP = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, step=1, grad_scale=1.0, scalars=None, seed=0, stream=None)


def entry(lib, **change):
    base = dict(param=P, master=P, grad=P, avg=P, sq=P, avg_scales=P, root_scales=P, n=128, weight_decay=0.1, param_bf16=1,
                grad_bf16=0)
    return lib._AdamwTensor(*(dict(base, **change).values()))


@pytest.mark.parametrize("change,status", [
    (dict(param=None), ENULL), (dict(grad=None), ENULL), (dict(avg=None), ENULL), (dict(sq=None), ENULL),
    (dict(avg_scales=None), ENULL), (dict(root_scales=None), ENULL), (dict(n=-1), ESHAPE), (dict(n=1 << 32), ESHAPE),
    (dict(param_bf16=0), EFLAG), (dict(param_bf16=2, master=None), EFLAG), (dict(grad_bf16=-1), EFLAG),
    (dict(param=P + 4), EALIGN), (dict(master=P + 4), EALIGN), (dict(grad=P + 4), EALIGN), (dict(avg=P + 4), EALIGN),
    (dict(sq=P + 8), EALIGN), (dict(avg_scales=P + 2), EALIGN), (dict(root_scales=P + 2), EALIGN),
])
def test_adamw_tensor_refusals(lib, change, status):
    # the bad tensor last: nothing may be enqueued for the good ones before it (there is no GPU here to enqueue on)
    table = (lib._AdamwTensor * 2)(entry(lib, n=0), entry(lib, **change))
    assert lib.raw.fp8bs_adamw_step(table, 2, *STEP.values()) == status


@pytest.mark.parametrize("change,status", [
    (dict(beta1=1.0), EFLAG), (dict(beta1=-0.1), EFLAG), (dict(beta2=1.0), EFLAG), (dict(beta2=float("nan")), EFLAG),
    (dict(eps=-1.0), EFLAG), (dict(eps=float("nan")), EFLAG), (dict(step=0), EFLAG), (dict(scalars=P + 2), EALIGN)])
def test_adamw_number_refusals(lib, change, status):
    table = (lib._AdamwTensor * 1)(entry(lib))
    assert lib.raw.fp8bs_adamw_step(table, 1, *dict(STEP, **change).values()) == status


def test_adamw_counts(lib):
    f = lib.raw.fp8bs_adamw_step
    table = (lib._AdamwTensor * 2)(entry(lib, n=0, param=None), entry(lib, n=0))
    assert f(table, -1, *STEP.values()) == ESHAPE
    assert f(None, 1, *STEP.values()) == ENULL
    assert f(None, 0, *STEP.values()) == OK
    assert f(table, 2, *STEP.values()) == OK          # tensors without elements


def test_struct_layout(lib):
    """The binding's structure as the header's is laid out: eight 8-byte fields, three of 4 bytes, padded to 8."""
    assert ctypes.sizeof(lib._AdamwTensor) == 80
    assert lib._AdamwTensor.n.offset == 56 and lib._AdamwTensor.grad_bf16.offset == 72


def test_binding_takes_only_device_tensors(lib):
    x = torch.zeros(4, 128, dtype=torch.uint8)
    s = torch.zeros(4, 1)
    with pytest.raises(TypeError):
        lib.fp8bs_gemm_gated(x, s, x, s)
    with pytest.raises(TypeError):
        lib.fp8bs_grouped_gemm_gated_ragged(x, s, torch.zeros(2, dtype=torch.int32), x, s)
    with pytest.raises(TypeError):
        lib.fp8bs_gated_backward(s.bfloat16(), s.bfloat16())
    with pytest.raises(TypeError):
        lib.fp8bs_adamw_table([s], [s], [s], [s])
    with pytest.raises(ValueError):
        lib.fp8bs_adamw_table([s], [s], [s], [])
    with pytest.raises(TypeError):
        lib.fp8bs_adamw_step([s], 1e-3, 1)
    empty = lib.fp8bs_adamw_table([], [], [], [])
    lib.fp8bs_adamw_step(empty, 1e-3, 1)
    with pytest.raises(ValueError):
        lib.fp8bs_adamw_step(empty, 1e-3, 1, seed=-1)
