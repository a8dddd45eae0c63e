"""A gated feed-forward block, and a mixture of gated experts, through a whole training step of the library: quantizers,
gated forward, down projection, its gradients, gated backward, activation and weight gradients, the optimizer step and the
weights' new codes.

Each operator's result is compared with 64 bits computed from what the step itself handed to it, so every connection
(which rows, which half of the stacked weight, which orientation, which scales) is checked and each bound is that of one
operator (linear_util, gated_util)."""

import pytest
import torch

from tests.gated_util import adamw64, backward64, check_codes, check_root_codes, gated64, random20
from tests.linear_util import ACTS, blocks64, check, gen, normal, product64, rows64

pytestmark = pytest.mark.gpu
HYPER = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8)


def host(*tensors):
    return [t.cpu() for t in tensors]


def wgrad_check(got, qa, sa, qb, sb, label):
    """f32 dW = A B^T of tiles along the tokens: the matrix core's own summation 2^-10, one rounding per block, two scales."""
    a, b = rows64(*host(qa, sa)), rows64(*host(qb, sb))
    mag = a.abs() @ b.abs().t()
    check(got, a @ b.t(), (2.0 ** -10 + (qa.shape[1] // 128 + 3) * 2.0 ** -24) * mag, label, bf16=False)


class Weight:
    """A weight under training: bf16, FP32 master, states in 8 bits, its gradient and its codes."""

    def __init__(self, lib, g, *shape):
        w = normal(g, *shape) * 0.05
        self.lib, self.p, self.master = lib, w.bfloat16().cuda(), w.cuda()
        n = w.numel()
        self.avg, self.root = (torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in range(2))
        self.avg_scale, self.root_scale = (torch.zeros(-(-n // 128), device="cuda") for _ in range(2))
        self.grad = torch.zeros(shape, device="cuda")
        self.code()

    def code(self):
        self.q, self.s = self.lib.fp8bs_quantize_w_128x128(self.p)

    def check_step(self, before, step, seed, number, label):
        p64, m64, v64, ep, em, ev = adamw64(before.flatten(), self.grad.cpu().flatten(), torch.zeros(before.numel()),
                                            torch.zeros(before.numel()), step=step, decay=0.1, **HYPER)
        check(self.master.flatten(), p64, ep, f"{label}: master", bf16=False)
        assert torch.equal(self.p, self.master.bfloat16())
        check_codes(self.avg.view(1, -1), self.avg_scale.view(1, -1), m64.view(1, -1), em.view(1, -1), f"{label}: m")
        r64 = v64.sqrt()
        er = torch.where(r64 > 0, ev / (2 * r64.clamp(min=1e-300)), torch.zeros_like(r64)) + 2.0 ** -23 * r64
        check_root_codes(self.root, self.root_scale, r64, er, random20(seed, step, number, r64.numel()), f"{label}: root")


def step_weights(lib, weights, seed):
    """One optimizer step over the weights, checked, and their new codes."""
    before = [w.master.cpu().clone() for w in weights]
    of = lambda name: [getattr(w, name) for w in weights]  # noqa: E731
    table = lib.fp8bs_adamw_table(of("p"), of("grad"), of("avg"), of("root"), master=of("master"), avg_scales=of("avg_scale"),
                                  root_scales=of("root_scale"), weight_decay=0.1)
    lib.fp8bs_adamw_step(table, step=1, seed=seed, **HYPER)
    torch.cuda.synchronize()
    for i, (w, b) in enumerate(zip(weights, before)):
        w.check_step(b, 1, seed, i, f"weight {i}")
        old = w.q.clone()
        w.code()
        assert not torch.equal(old, w.q)


@pytest.mark.parametrize("tokens,d,n,act", [(128, 256, 128, "silu"), (384, 512, 256, "gelu_tanh"), (2048, 256, 1152, "silu")])
def test_dense_training_step(gpu_lib, tokens, d, n, act):
    lib, g = gpu_lib, gen(tokens + n)
    x = normal(g, tokens, d).bfloat16().cuda()
    up, down = Weight(lib, g, 2 * n, d), Weight(lib, g, d, n)

    # ---- forward
    xq, xs, xqt, xst = lib.fp8bs_quantize_act_1x128_dual(x)
    z = torch.empty((tokens, 2 * n), dtype=torch.bfloat16, device="cuda")
    _, hq, hs = lib.fp8bs_gemm_gated(xq, xs, up.q, up.s, act=ACTS[act], z=z, h=False, qh=None)
    y = lib.fp8bs_gemm(hq, hs, down.q, down.s)
    z64, ez, h64, eh = gated64(*host(xq, xs, up.q, up.s), act)
    check(z, z64, ez, "z")
    check_codes(hq, hs, h64, eh, "h")
    check(y, *product64(*host(hq, hs, down.q, down.s), 0), "y")

    # ---- backward of sum(y * v)
    v = (normal(g, tokens, d) * 0.1).bfloat16().cuda()
    vq, vs, vqt, vst = lib.fp8bs_quantize_act_1x128_dual(v)
    dh = lib.fp8bs_gemm(vq, vs, down.q, down.s, b_layout=1)
    _, q, s, qt, st, _, hqt, hst = lib.fp8bs_gated_backward(dh, z, act=ACTS[act], dz=False, q=None, qt=None, qht=None)
    dx = lib.fp8bs_gemm(q, s, up.q, up.s, b_layout=1)
    lib.fp8bs_gemm_wgrad(qt, st, xqt, xst, c=up.grad)
    lib.fp8bs_gemm_wgrad(vqt, vst, hqt, hst, c=down.grad)
    torch.cuda.synchronize()
    check(dh, *product64(*host(vq, vs, down.q, down.s), 1), "dh")
    w = backward64(*host(dh, z), act)
    both = [torch.cat([w["dg"][i], w["du"][i]], 1) for i in (0, 1)]
    check_codes(q, s, *both, "dz along the columns")
    check_codes(qt, st, both[0].t().contiguous(), both[1].t().contiguous(), "dz along the rows")
    check_codes(hqt, hst, w["h"][0].t().contiguous(), w["h"][1].t().contiguous(), "h along the rows")
    check(dx, *product64(*host(q, s, up.q, up.s), 1), "dx")
    wgrad_check(up.grad, qt, st, xqt, xst, "gate and up gradient")
    wgrad_check(down.grad, vqt, vst, hqt, hst, "down gradient")
    # the whole backward pass against autograd on the values that the codes stand for: what lies between are the
    # codes of v, dh, dz (2^-4 of a value each, random signs) and the bf16 of z and dh: within a tenth in norm
    xv, wu, wd = rows64(*host(xq, xs)).requires_grad_(), blocks64(*host(up.q, up.s)), blocks64(*host(down.q, down.s))
    zz = xv @ wu.t()
    gate = zz[:, :n]
    a = torch.nn.functional.silu(gate) if act == "silu" else torch.nn.functional.gelu(gate, approximate="tanh")
    ((a * zz[:, n:]) @ wd.t() * v.double().cpu()).sum().backward()
    assert float((dx.double().cpu() - xv.grad).norm() / xv.grad.norm()) < 0.1

    step_weights(lib, [up, down], seed=tokens)


@pytest.mark.parametrize("tokens,topk,experts", [(3, 2, 6), (200, 3, 8), (1500, 4, 6)])
def test_experts_training_step(gpu_lib, tokens, topk, experts):
    lib, g = gpu_lib, gen(tokens)
    d, n, act = 256, 384, "silu"
    ids = torch.stack([torch.randperm(experts, generator=g)[:topk] for _ in range(tokens)]).int()
    ids[torch.rand(ids.shape, generator=g) < 0.1] = -1                       # dropped pairs: rows behind the last segment
    gates = torch.rand((tokens, topk), generator=g)
    x = normal(g, tokens, d).bfloat16().cuda()
    up, down = Weight(lib, g, experts, 2 * n, d), Weight(lib, g, experts, d, n)

    # ---- forward
    seg, slot, tok = lib.fp8bs_moe_route_ragged(ids.cuda(), experts)
    rows, total = tokens * topk, int((ids >= 0).sum())
    q, s = torch.zeros((rows, d), dtype=torch.uint8, device="cuda"), torch.zeros((rows, d // 128), device="cuda")
    lib.fp8bs_moe_permute_quantize(x, slot, seg, tok, q=q, scales=s)
    z = torch.full((rows, 2 * n), 2.0, dtype=torch.bfloat16, device="cuda")
    hq, hs = torch.full((rows, n), 0x5A, dtype=torch.uint8, device="cuda"), torch.full((rows, n // 128), 3.0, device="cuda")
    lib.fp8bs_grouped_gemm_gated_ragged(q, s, seg, up.q, up.s, act=ACTS[act], z=z, h=False, qh=hq, sh=hs)
    y = torch.zeros((rows, d), dtype=torch.bfloat16, device="cuda")
    lib.fp8bs_grouped_gemm_ragged(hq, hs, seg, down.q, down.s, c=y)
    out = lib.fp8bs_moe_combine(y, slot, gates.cuda())
    torch.cuda.synchronize()
    cuts = [slice(a, b) for a, b in zip(seg.tolist(), seg.tolist()[1:])]
    assert int(seg[-1]) == total and (z[total:] == 2.0).all() and (hq[total:] == 0x5A).all() and (hs[total:] == 3.0).all()
    for e, cut in enumerate(cuts):
        if cut.start < cut.stop:
            z64, ez, h64, eh = gated64(*host(q[cut], s[cut], up.q[e], up.s[e]), act)
            check(z[cut], z64, ez, f"z of {e}")
            check_codes(hq[cut], hs[cut], h64, eh, f"h of {e}")
            check(y[cut], *product64(*host(hq[cut], hs[cut], down.q[e], down.s[e]), 0), f"y of {e}")
    assert torch.isfinite(out).all()

    # ---- backward of sum(out * v)
    v = (normal(g, tokens, d) * 0.1).bfloat16().cuda()
    gate_rows = torch.zeros(rows, device="cuda")
    at = slot.flatten().long()
    gate_rows[at[at >= 0]] = gates.cuda().flatten()[at >= 0]
    dy = torch.zeros((rows, d), dtype=torch.bfloat16, device="cuda")
    dy[:total] = (v[tok[:total].long()].float() * gate_rows[:total, None]).bfloat16()
    xr = torch.zeros((rows, d), dtype=torch.bfloat16, device="cuda")
    xr[:total] = x[tok[:total].long()]
    dyq, dys = lib.fp8bs_quantize_act_1x128(dy)
    dh = lib.fp8bs_grouped_gemm_ragged(dyq, dys, seg, down.q, down.s, b_layout=1)
    dz, dzq, dzs, _, _, h, _, _ = lib.fp8bs_gated_backward(dh, z, act=ACTS[act], q=None, h=None, row_end=seg[-1:])
    dxr = lib.fp8bs_grouped_gemm_ragged(dzq, dzs, seg, up.q, up.s, b_layout=1)
    lib.fp8bs_grouped_wgrad_ragged(dz, xr, seg, c=up.grad)
    lib.fp8bs_grouped_wgrad_ragged(dy, h, seg, c=down.grad)
    dx = lib.fp8bs_moe_combine(dxr, slot, (slot >= 0).float())
    torch.cuda.synchronize()
    w = backward64(*host(dh[:total], z[:total]), act)
    both = [torch.cat([w["dg"][i], w["du"][i]], 1) for i in (0, 1)]
    check(dz[:total], *both, "dz")
    check(h[:total], *w["h"], "h again")
    check_codes(dzq[:total], dzs[:total], *both, "dz codes")
    for e, cut in enumerate(cuts):
        for got, a, b, label in ((up.grad[e], dz[cut], xr[cut], "gate and up"), (down.grad[e], dy[cut], h[cut], "down")):
            a, b = a.double().cpu(), b.double().cpu()
            check(got, a.t() @ b, 2.0 ** -23 * (cut.stop - cut.start + 2) * (a.abs().t() @ b.abs()), f"{label} of {e}", bf16=False)
        if cut.start < cut.stop:
            check(dxr[cut], *product64(*host(dzq[cut], dzs[cut], up.q[e], up.s[e]), 1), f"dx rows of {e}")
    assert torch.isfinite(dx).all()
    step_weights(lib, [up, down], seed=tokens)


def test_dense_step_in_one_graph(gpu_lib):
    """The step from the activation's codes to the optimizer, captured: every replay equals eager steps from the same state."""
    lib, g = gpu_lib, gen(7)
    tokens, d, n = 256, 256, 256
    x, v = normal(g, tokens, d).bfloat16().cuda(), (normal(g, tokens, d) * 0.1).bfloat16().cuda()
    sides = []
    for _ in range(2):
        h = gen(8)
        sides.append((Weight(lib, h, 2 * n, d), Weight(lib, h, d, n)))
    scalars = torch.tensor([1e-3, 1.0, 1.0], device="cuda")

    def program(up, down):
        """Buffers, and the step on them."""
        bf = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        u8 = lambda *s: torch.empty(s, dtype=torch.uint8, device="cuda")  # noqa: E731
        f = lambda *s: torch.empty(s, device="cuda")  # noqa: E731
        xd = lib.fp8bs_quantize_act_1x128_dual(x)
        vd = lib.fp8bs_quantize_act_1x128_dual(v)
        z, hq, hs, y, dh = bf(tokens, 2 * n), u8(tokens, n), f(tokens, n // 128), bf(tokens, d), bf(tokens, n)
        ws = f(max(4, lib.fp8bs_gemm_gated_workspace(tokens, n, d) // 4))
        q, s, qt, st = u8(tokens, 2 * n), f(tokens, 2 * n // 128), u8(2 * n, tokens), f(2 * n, tokens // 128)
        hqt, hst = u8(n, tokens), f(n, tokens // 128)
        of = lambda name: [up.__dict__[name], down.__dict__[name]]  # noqa: E731
        table = lib.fp8bs_adamw_table(of("p"), of("grad"), of("avg"), of("root"), master=of("master"),
                                      avg_scales=of("avg_scale"), root_scales=of("root_scale"), weight_decay=0.1)

        def step():
            for w in (up, down):
                lib.fp8bs_quantize_w_128x128(w.p, q=w.q, scales=w.s)
            lib.fp8bs_gemm_gated(xd[0], xd[1], up.q, up.s, z=z, h=False, qh=hq, sh=hs, workspace=ws)
            lib.fp8bs_gemm(hq, hs, down.q, down.s, c=y)
            lib.fp8bs_gemm(vd[0], vd[1], down.q, down.s, b_layout=1, c=dh)
            lib.fp8bs_gated_backward(dh, z, dz=False, q=q, scales=s, qt=qt, scales_t=st, qht=hqt, scales_ht=hst)
            lib.fp8bs_gemm_wgrad(qt, st, xd[2], xd[3], c=up.grad)
            lib.fp8bs_gemm_wgrad(vd[2], vd[3], hqt, hst, c=down.grad)
            lib.fp8bs_adamw_step(table, 0.0, 0, scalars=scalars, seed=3)

        return step, y

    eager, ye = program(*sides[0])
    captured, yc = program(*sides[1])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured()
    for i in range(1, 5):
        scalars.copy_(torch.tensor([1e-3 / i, 1.0, float(i)]))
        eager()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(ye, yc)
        for a, b in zip(*sides):
            for name in ("p", "master", "avg", "root", "avg_scale", "root_scale", "grad", "q", "s"):
                assert torch.equal(getattr(a, name), getattr(b, name)), (i, name)
