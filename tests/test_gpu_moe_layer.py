"""A mixture-of-experts layer with its dense shared expert, forward and backward, through the library: the unpadded
routing, the ragged expert products and weight gradients, the linear layer's epilogue and its backward pass, with the
quantizers, the dispatch and the combine between them.

Each product is compared with 64 bits computed from the codes and bf16 values that the layer itself handed to it, so
every connection (which rows, which weights, which scales, which residual) is checked and each bound is that of one
operator (linear_util).  The layer's own loss is checked against differences in a last test, without FP8 codes in the
way of a derivative: the expert weights' gradient, which is taken from bf16 rows.
"""

import pytest
import torch

from tests.linear_util import (ACTS, SLOPE, act64, argument, blocks, check, gen, normal, product64)

pytestmark = pytest.mark.gpu


def split(seg):
    s = seg.tolist()
    return [slice(a, b) for a, b in zip(s, s[1:])]


@pytest.mark.parametrize("tokens,topk,experts", [(1, 2, 8), (7, 3, 40), (300, 4, 10), (2500, 4, 6)])
def test_layer_forward_and_backward(gpu_lib, tokens, topk, experts):
    lib, g = gpu_lib, gen(tokens + experts)
    h, f = 256, 384
    ids = torch.stack([torch.randperm(experts, generator=g)[:topk] for _ in range(tokens)]).int()
    ids[torch.rand(ids.shape, generator=g) < 0.1] = -1                       # dropped pairs
    gates = torch.rand((tokens, topk), generator=g)
    x = normal(g, tokens, h).bfloat16().cuda()
    up_q, up_s = (t.cuda() for t in blocks(normal(g, experts, h, h) * 0.05))
    w1q, w1s = (t.cuda() for t in blocks(normal(g, f, h) * 0.05))
    w2q, w2s = (t.cuda() for t in blocks(normal(g, h, f) * 0.05))
    b1, b2 = normal(g, f).cuda(), normal(g, h).cuda()

    # ---- forward
    seg, slot, tok = lib.fp8bs_moe_route_ragged(ids.cuda(), experts)
    rows = tokens * topk
    q, s = torch.zeros((rows, h), dtype=torch.uint8, device="cuda"), torch.zeros((rows, h // 128), device="cuda")
    lib.fp8bs_moe_permute_quantize(x, slot, seg, tok, q=q, scales=s)
    y = torch.full((rows, h), 3.0, dtype=torch.bfloat16, device="cuda")
    lib.fp8bs_grouped_gemm_ragged(q, s, seg, up_q, up_s, c=y)
    routed = lib.fp8bs_moe_combine(y, slot, gates.cuda())
    xq, xs = lib.fp8bs_quantize_act_1x128(x)
    z = torch.empty((tokens, f), dtype=torch.bfloat16, device="cuda")
    hid = lib.fp8bs_gemm_epilogue(xq, xs, w1q, w1s, bias=b1, act=ACTS["silu"], z=z)
    hq, hs = lib.fp8bs_quantize_act_1x128(hid)
    out = lib.fp8bs_gemm_epilogue(hq, hs, w2q, w2s, bias=b2, residual=routed)
    torch.cuda.synchronize()

    cuts, total = split(seg), int(seg[-1])
    assert total == int((ids >= 0).sum())
    assert torch.equal(q[:total], xq[tok[:total].long()]) and torch.equal(s[:total], xs[tok[:total].long()])
    assert (tok[total:] == -1).all() and (y[total:] == 3.0).all()
    for e, cut in enumerate(cuts):
        if cut.start < cut.stop:
            w, err = product64(q[cut].cpu(), s[cut].cpu(), up_q[e].cpu(), up_s[e].cpu(), 0)
            check(y[cut], w, err, f"expert {e}")
    z64, ez = product64(xq.cpu(), xs.cpu(), w1q.cpu(), w1s.cpu(), 0)
    z64 = z64 + b1.double().cpu()
    ez = ez + 2.0 ** -24 * (z64.abs() + ez)
    check(z, z64, ez, "z")
    check(hid, act64(z64, "silu"), SLOPE * ez + (argument(z64, "silu") + 4) * 2.0 ** -24 * z64.abs(), "hidden")
    o64, eo = product64(hq.cpu(), hs.cpu(), w2q.cpu(), w2s.cpu(), 0)
    o64 = o64 + b2.double().cpu() + routed.double().cpu()
    check(out, o64, eo + 2 * 2.0 ** -24 * (o64.abs() + eo), "out")

    # ---- backward of sum(out * v)
    v = (normal(g, tokens, h) * 0.1).bfloat16().cuda()
    _, db2 = lib.fp8bs_epilogue_backward(v, None, dz=False)
    vq, vs = lib.fp8bs_quantize_act_1x128(v)
    dh = lib.fp8bs_gemm_epilogue(vq, vs, w2q, w2s, b_layout=1)
    dz, db1 = lib.fp8bs_epilogue_backward(dh, z, act=ACTS["silu"])
    # routed part: each expert row gets gate * v of its token
    live = tok[:total].long()
    gate_rows = torch.zeros(rows, device="cuda")
    at = slot.flatten().long()
    gate_rows[at[at >= 0]] = gates.cuda().flatten()[at >= 0]
    dy = torch.zeros((rows, h), dtype=torch.bfloat16, device="cuda")
    dy[:total] = (v[live].float() * gate_rows[:total, None]).bfloat16()
    xr = torch.zeros((rows, h), dtype=torch.bfloat16, device="cuda")
    xr[:total] = x[live]
    dw = lib.fp8bs_grouped_wgrad_ragged(dy, xr, seg)
    dyq, dys = lib.fp8bs_quantize_act_1x128(dy)
    dxr = lib.fp8bs_grouped_gemm_ragged(dyq, dys, seg, up_q, up_s, b_layout=1)
    routed_dx = lib.fp8bs_moe_combine(dxr, slot, (slot >= 0).float())
    dzq, dzs = lib.fp8bs_quantize_act_1x128(dz)
    dx = lib.fp8bs_gemm_epilogue(dzq, dzs, w1q, w1s, b_layout=1, residual=routed_dx)
    torch.cuda.synchronize()

    check(db2, v.double().cpu().sum(0), tokens * 2.0 ** -24 * v.double().cpu().abs().sum(0), "db2", bf16=False)
    p64, ep = product64(vq.cpu(), vs.cpu(), w2q.cpu(), w2s.cpu(), 1)
    check(dh, p64, ep, "dh")
    # dz and db1 against differences of the loss through act, at the bf16 z and dh that the call was given
    zd, dhd, step = z.double().cpu(), dh.double().cpu(), 1e-5
    diff = (act64(zd + step, "silu") - act64(zd - step, "silu")) / (2 * step) * dhd
    # differences: h^2 / 6 of a third derivative below 3 and 2^-52 |act| / h of cancellation; slope: see linear_util
    e = dhd.abs() * (step * step + 2.0 ** -50 * zd.abs() / step + (2 * argument(zd, "silu") + 8) * 2.0 ** -24 * (1 + zd.abs()))
    check(dz, diff, e, "dz")
    check(db1, diff.sum(0), e.sum(0) + tokens * 2.0 ** -24 * (diff.abs() + e).sum(0), "db1", bf16=False)
    for i, cut in enumerate(cuts):
        a, b = dy[cut].double().cpu(), xr[cut].double().cpu()
        check(dw[i], a.t() @ b, 2.0 ** -23 * (cut.stop - cut.start + 2) * (a.abs().t() @ b.abs()), f"dw {i}", bf16=False)
        if cut.start < cut.stop:
            w, err = product64(dyq[cut].cpu(), dys[cut].cpu(), up_q[i].cpu(), up_s[i].cpu(), 1)
            check(dxr[cut], w, err, f"dx rows of {i}")
    d64, ed = product64(dzq.cpu(), dzs.cpu(), w1q.cpu(), w1s.cpu(), 1)
    d64 = d64 + routed_dx.double().cpu()
    check(dx, d64, ed + 2.0 ** -24 * (d64.abs() + ed), "dx")


def test_weight_gradient_against_differences(gpu_lib):
    """dW of L = sum_t sum_i v[t, i] (W_e x_t)_i over ragged segments: L's central difference in single weights."""
    g = gen(5)
    lengths, m, n = [3, 0, 17], 16, 24
    seg = torch.tensor([0, 3, 3, 20], dtype=torch.int32)
    v, x = normal(g, 20, m).bfloat16(), normal(g, 20, n).bfloat16()
    dw = gpu_lib.fp8bs_grouped_wgrad_ragged(v.cuda(), x.cuda(), seg.cuda()).cpu().double()
    w = normal(g, 3, m, n).double()

    def loss(w):
        return sum((v[a:b].double() * (x[a:b].double() @ w[e].t())).sum()
                   for e, (a, b) in enumerate(zip(seg.tolist(), seg.tolist()[1:])))

    for e, i, j in ((0, 0, 0), (0, 15, 23), (1, 4, 4), (2, 7, 11), (2, 0, 23)):
        up, down = w.clone(), w.clone()
        up[e, i, j] += 0.5
        down[e, i, j] -= 0.5
        diff = float(loss(up) - loss(down))                      # L is linear: exact but for 2^-52 of its terms
        mag = float((v.double().abs()[:, i] * x.double().abs()[:, j]).sum())
        assert abs(float(dw[e, i, j]) - diff) <= 2.0 ** -23 * 22 * mag + 1e-10, (e, i, j)
