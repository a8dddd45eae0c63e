"""The optimizer step on the GPU against its 64-bit form (gated_util)."""

import pytest
import torch

from tests.gated_util import E4M3, adamw64, check_codes, check_root_codes, random20
from tests.linear_util import check, gen, normal

pytestmark = pytest.mark.gpu
HYPER = dict(lr=3e-3, beta1=0.9, beta2=0.95, eps=1e-8)


class Case:
    """One tensor of an optimizer table, on the host and on the device."""

    def __init__(self, g, n, eight=False, bf16=False, master=False, grad_bf16=False, decay=0.1, fresh=False):
        self.n, self.eight, self.decay = n, eight, decay
        w = normal(g, n) * 0.02
        self.p = w.bfloat16() if bf16 else w
        self.master = w.clone() if master else None
        grad = normal(g, n) * 1e-3 * torch.exp(normal(g, n))
        self.g = grad.bfloat16() if grad_bf16 else grad
        m = torch.zeros(n) if fresh else normal(g, n) * 3e-4
        r = torch.zeros(n) if fresh else normal(g, n).abs() * 1e-3 + 1e-6
        groups = -(-n // 128)
        if eight:
            self.m, self.ms = self.code(m, groups)
            self.v, self.rs = self.code(r, groups)
        else:
            self.m, self.v, self.ms, self.rs = m, r * r, None, None
        self.to_device()

    @staticmethod
    def code(x, groups):
        t = torch.cat([x, x.new_zeros(groups * 128 - x.numel())]).view(groups, 128)
        s = t.abs().amax(1) / 448.0
        q = (t / s.clamp(min=1e-30)[:, None]).clamp(-448, 448).to(E4M3).view(torch.uint8).view(-1)[:x.numel()]
        return q.contiguous(), s

    def to_device(self):
        on = lambda t: None if t is None else t.cuda().contiguous()  # noqa: E731
        self.dp, self.dw, self.dg, self.dm, self.dv = on(self.p), on(self.master), on(self.g), on(self.m), on(self.v)
        self.dms, self.drs = on(self.ms), on(self.rs)

    def states(self):
        """m and v in FP32, as the kernel reads them."""
        if not self.eight:
            return self.m, self.v
        spread = lambda s: s.repeat_interleave(128)[:self.n]  # noqa: E731
        r = self.v.view(E4M3).float() * spread(self.rs)
        return self.m.view(E4M3).float() * spread(self.ms), r * r

    def check(self, label, step, seed, number, grad_scale=1.0, **hyper):
        m, v = self.states()
        p = self.master if self.master is not None else self.p.float()
        p64, m64, v64, ep, em, ev = adamw64(p, self.g.float(), m, v, step=step, decay=self.decay, grad_scale=grad_scale, **hyper)
        check(self.dp, p64, ep, f"{label}: p", bf16=self.p.dtype == torch.bfloat16)
        if self.master is not None:
            check(self.dw, p64, ep, f"{label}: master", bf16=False)
            assert torch.equal(self.dw.bfloat16(), self.dp), f"{label}: p is the master rounded"
        if not self.eight:
            check(self.dm, m64, em, f"{label}: m", bf16=False)
            check(self.dv, v64, ev, f"{label}: v", bf16=False)
            return
        pad = (-self.n) % 128
        wide = lambda t: torch.cat([t, t.new_zeros(pad)]).view(1, -1)  # noqa: E731
        check_codes(wide(self.dm.cpu()), self.dms.view(1, -1), wide(m64), wide(em), f"{label}: m")
        r64 = v64.sqrt()
        er = torch.where(r64 > 0, ev / (2 * r64.clamp(min=1e-300)), torch.zeros_like(r64)) + 2.0 ** -23 * r64
        check_root_codes(self.dv, self.drs, r64, er, random20(seed, step, number, self.n), f"{label}: root")


def table_of(lib, cases):
    of = lambda name: [getattr(c, name) for c in cases]  # noqa: E731
    return lib.fp8bs_adamw_table(of("dp"), of("dg"), of("dm"), of("dv"), master=of("dw"), avg_scales=of("dms"),
                                 root_scales=of("drs"), weight_decay=of("decay"))


KINDS = [dict(), dict(bf16=True), dict(bf16=True, master=True), dict(bf16=True, master=True, grad_bf16=True), dict(grad_bf16=True)]


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("kind", range(len(KINDS)))
@pytest.mark.parametrize("n", [1, 3, 127, 128, 130, 4095, 4096, 4099, 70001])
def test_one_tensor(gpu_lib, n, kind, eight):
    c = Case(gen(n + kind), n, eight=eight, **KINDS[kind])
    gpu_lib.fp8bs_adamw_step(table_of(gpu_lib, [c]), step=7, seed=5, **HYPER)
    torch.cuda.synchronize()
    c.check("tensor", 7, 5, 0, **HYPER)


@pytest.mark.parametrize("step,eight", [(1, False), (1, True), (100000, True)])
def test_first_and_late_steps(gpu_lib, step, eight):
    c = Case(gen(step), 5000, eight=eight, bf16=True, master=True, fresh=step == 1)
    gpu_lib.fp8bs_adamw_step(table_of(gpu_lib, [c]), step=step, seed=1 << 31, grad_scale=0.25, **HYPER)
    c.check("step", step, 1 << 31, 0, grad_scale=0.25, **HYPER)


def test_many_tensors_of_mixed_kinds(gpu_lib):
    """More than a launch takes, sizes from none to many workgroups, kinds in turn; what lies between them stays."""
    g = gen(77)
    sizes = [0, 1, 129, 5000, 128, 4096, 0, 12345, 77, 256]
    cases = [Case(g, sizes[i % 10], eight=i % 7 > 2, decay=0.01 * (i % 3), **KINDS[i % 5]) for i in range(103)]
    gpu_lib.fp8bs_adamw_step(table_of(gpu_lib, cases), step=3, seed=99, **HYPER)
    torch.cuda.synchronize()
    for i, c in enumerate(cases):
        if c.n:
            c.check(f"tensor {i}", 3, 99, i, **HYPER)


def test_views_of_flat_storage(gpu_lib):
    """Tensors side by side in one buffer, with gaps: the gaps keep what they held."""
    g, sizes = gen(5), [200, 128, 1, 999]
    flat = {k: torch.full((4096,), 7.0, device="cuda") for k in ("p", "g", "m", "v")}
    views, at = {k: [] for k in flat}, 0
    for n in sizes:
        for k in flat:
            views[k].append(flat[k][at:at + n])
        at += -(-n // 128) * 128
    for k in flat:
        for t in views[k]:
            t.copy_(normal(g, t.numel()).abs() * 1e-2)
    before = {k: v.clone() for k, v in flat.items()}
    gpu_lib.fp8bs_adamw_step(gpu_lib.fp8bs_adamw_table(views["p"], views["g"], views["m"], views["v"]), 1e-3, 2)
    own = torch.zeros(4096, dtype=torch.bool, device="cuda")
    at = 0
    for n in sizes:
        own[at:at + n] = True
        at += -(-n // 128) * 128
    for k in flat:
        assert torch.equal(flat[k][~own], before[k][~own])
    assert torch.equal(flat["g"], before["g"]) and not torch.equal(flat["p"][own], before["p"][own])


@pytest.mark.parametrize("n", [1, 126, 127, 129, 1023, 1025, 4001])
def test_nothing_behind_the_end(gpu_lib, n):
    """8-bit states, bf16 parameters and gradients in the middle of larger buffers: the rest keeps what it held."""
    groups = -(-n // 128)
    make = lambda t, k: torch.full((k + 512,), 3, dtype=t, device="cuda")  # noqa: E731
    sizes = {"p": (torch.bfloat16, n), "w": (torch.float32, n), "g": (torch.bfloat16, n), "m": (torch.uint8, n),
             "r": (torch.uint8, n), "ms": (torch.float32, groups), "rs": (torch.float32, groups)}
    buffers = {k: make(*v) for k, v in sizes.items()}
    views = {k: buffers[k][256:256 + v[1]] for k, v in sizes.items()}
    table = gpu_lib.fp8bs_adamw_table([views["p"]], [views["g"]], [views["m"]], [views["r"]], master=[views["w"]],
                                      avg_scales=[views["ms"]], root_scales=[views["rs"]])
    gpu_lib.fp8bs_adamw_step(table, 0.5, 1)
    torch.cuda.synchronize()
    for k, b in buffers.items():
        assert (b[:256] == 3).all() and (b[256 + sizes[k][1]:] == 3).all(), k
        assert k == "g" or not (views[k] == 3).all(), k
    assert (views["g"] == 3).all()


def test_rounding_at_random(gpu_lib):
    """Over many seeds the mean of r's codes nears r: half of 1/sqrt(seeds) of a step, times 6; two seeds differ,
    one seed twice does not."""
    n, seeds = 1280, 256
    base = Case(gen(3), n, eight=True)
    total, first = torch.zeros(n, dtype=torch.float64), None
    for seed in range(seeds):
        c = Case(gen(3), n, eight=True)
        gpu_lib.fp8bs_adamw_step(table_of(gpu_lib, [c]), step=10, seed=seed, **HYPER)
        r = c.dv.cpu().view(E4M3).double() * c.drs.cpu().double().repeat_interleave(128)[:n]
        total += r
        if seed == 0:
            first = c.dv.clone()
        elif seed == 1:
            assert not torch.equal(first, c.dv)
    again = Case(gen(3), n, eight=True)
    gpu_lib.fp8bs_adamw_step(table_of(gpu_lib, [again]), step=10, seed=0, **HYPER)
    assert torch.equal(first, again.dv)
    m, v = base.states()
    r64 = (0.95 * v.double() + 0.05 * base.g.double() ** 2).sqrt()
    step = torch.maximum(r64 / 8, 2.0 ** -9 * again.drs.cpu().double().repeat_interleave(128)[:n])
    assert ((total / seeds - r64).abs() <= 3.0 / seeds ** 0.5 * step + 2.0 ** -8 * step).all()


def test_zero_gradients_and_states(gpu_lib):
    c = Case(gen(1), 300, eight=True, fresh=True, decay=0.0)
    c.dg.zero_()
    p = c.dp.clone()
    gpu_lib.fp8bs_adamw_step(table_of(gpu_lib, [c]), step=1, **HYPER)
    assert torch.equal(c.dp, p) and not c.dm.any() and not c.dv.any() and not c.dms.any() and not c.drs.any()
    assert torch.isfinite(c.dp).all()


def test_small_gradients_beside_large_ones(gpu_lib):
    """A group that spans 2^40: no positive root becomes zero, so no update is larger than the second moment allows."""
    n = 256
    c = Case(gen(8), n, eight=True, fresh=True)
    c.g = torch.exp2(-40 * torch.rand(n, generator=gen(9)))
    c.to_device()
    gpu_lib.fp8bs_adamw_step(table_of(gpu_lib, [c]), step=1, **HYPER)
    c.check("wide group", 1, 0, 0, **HYPER)
    assert (c.dv & 0x7F).all()


def test_numbers_on_the_device_and_graphs(gpu_lib):
    """A captured step reads lr, grad_scale and step when it runs: every replay equals an eager step."""
    make = lambda: [Case(gen(21), 5001, eight=True, bf16=True, master=True), Case(gen(22), 333)]  # noqa: E731
    captured, eager = make(), make()
    scalars = torch.tensor([1e-3, 1.0, 1.0], device="cuda")
    table = table_of(gpu_lib, captured)
    state = [[t.clone() for t in (c.dp, c.dm, c.dv)] for c in captured]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gpu_lib.fp8bs_adamw_step(table, 0.0, 0, scalars=scalars, seed=4)
    for c, s in zip(captured, state):                 # capture runs nothing
        assert all(torch.equal(a, b) for a, b in zip((c.dp, c.dm, c.dv), s))
    etable = table_of(gpu_lib, eager)
    for step in range(1, 5):
        lr, scale = 1e-3 * step, 0.5 * step
        scalars.copy_(torch.tensor([lr, scale, float(step)]))
        graph.replay()
        torch.cuda.synchronize()
        gpu_lib.fp8bs_adamw_step(etable, 0.0, 0, scalars=torch.tensor([lr, scale, float(step)], device="cuda"), seed=4)
        torch.cuda.synchronize()
        for a, b in zip(captured, eager):
            for x, y in ((a.dp, b.dp), (a.dm, b.dm), (a.dv, b.dv), (a.dw, b.dw), (a.dms, b.dms), (a.drs, b.drs)):
                assert x is None or torch.equal(x, y)
    one = Case(gen(30), 2000, eight=True)
    gpu_lib.fp8bs_adamw_step(table_of(gpu_lib, [one]), 0.0, 0, scalars=torch.tensor([3e-3, 0.25, 12.0], device="cuda"), seed=6)
    one.check("device numbers", 12, 6, 0, grad_scale=0.25, **HYPER)


def test_table_refusals(gpu_lib):
    f = gpu_lib.fp8bs_adamw_table
    x = lambda n=128, t=torch.float32: torch.zeros(n, dtype=t, device="cuda")  # noqa: E731
    u8, bf = torch.uint8, torch.bfloat16
    with pytest.raises(ValueError):
        f([x()], [x(64)], [x()], [x()])
    with pytest.raises(TypeError):
        f([x(t=torch.float16)], [x()], [x()], [x()])
    with pytest.raises(TypeError):
        f([x()], [x(t=u8)], [x()], [x()])
    with pytest.raises(TypeError):
        f([x()], [x()], [x(t=u8)], [x()])
    with pytest.raises(TypeError):
        f([x()], [x()], [x()], [x()], avg_scales=[x(1)], root_scales=[x(1)])
    with pytest.raises(ValueError):
        f([x()], [x()], [x(t=u8)], [x(t=u8)], avg_scales=[x(1)], root_scales=None)
    with pytest.raises(ValueError):
        f([x(200)], [x(200)], [x(200, u8)], [x(200, u8)], avg_scales=[x(1)], root_scales=[x(1)])
    with pytest.raises(ValueError):
        f([x()], [x()], [x()], [x()], master=[x()])
    with pytest.raises(ValueError):
        f([x(256)[::2]], [x()], [x()], [x()])
    with pytest.raises(TypeError):
        f([x().cpu()], [x()], [x()], [x()])
    p, m, big = x(), x(), x(1024)
    with pytest.raises(ValueError):
        f([p, p], [x(), x()], [x(), x()], [x(), x()])
    with pytest.raises(ValueError):
        f([p], [x()], [m], [m])
    with pytest.raises(ValueError):
        f([p], [p], [x()], [x()])
    with pytest.raises(ValueError):
        f([big[:512], x()], [x(512), x()], [x(512), big[508:636]], [x(512), x()])
    g = x()
    f([p, x()], [g, g], [x(), x()], [m, x()])         # a shared gradient is read twice
    f([big[:512], big[512:]], [x(512), x(512)], [x(512), x(512)], [x(512), x(512)])
    odd = f([x(256)[1:129]], [x()], [x()], [x()])
    with pytest.raises(gpu_lib.Fp8bsError):
        gpu_lib.fp8bs_adamw_step(odd, 1e-3, 1)
    good = f([x(t=bf)], [x()], [x()], [x()])
    for bad in (dict(beta1=1.0), dict(eps=-1.0)):
        with pytest.raises(gpu_lib.Fp8bsError):
            gpu_lib.fp8bs_adamw_step(good, 1e-3, 1, **bad)
    with pytest.raises(gpu_lib.Fp8bsError):
        gpu_lib.fp8bs_adamw_step(good, 1e-3, 0)
    with pytest.raises(ValueError):
        gpu_lib.fp8bs_adamw_step(good, 1e-3, 1, scalars=x(2))
    torch.cuda.synchronize()


def test_other_stream(gpu_lib):
    a, b = Case(gen(41), 3001, eight=True), Case(gen(41), 3001, eight=True)
    gpu_lib.fp8bs_adamw_step(table_of(gpu_lib, [a]), step=2, **HYPER)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    gpu_lib.fp8bs_adamw_step(table_of(gpu_lib, [b]), step=2, stream=side, **HYPER)
    side.synchronize()
    torch.cuda.synchronize()
    for x, y in ((a.dp, b.dp), (a.dm, b.dm), (a.dv, b.dv), (a.dms, b.dms), (a.drs, b.drs)):
        assert torch.equal(x, y)


def test_several_steps_have_the_bits_of_tensor_operations(gpu_lib):
    """States in 8 bits after four steps against the same formulas in single FP32 operations: every one of them rounds
    alike, so the states' drift is the formulas' own.  A code may still differ where the kernel's quotient (within 2^-22 of
    a unit of the exact one before it rounds) is rounded to the other side, which in 2^19 elements, four
    steps, two states with a rounding boundary within such a distance of about one in 2^21 should happen about twice
    at most; a differing code may move its group's later scales, so groups are counted: at most 8 of 4096."""
    n, seed, lr, b1, b2, eps, decay = 1 << 19, 77, 1e-3, 0.9, 0.95, 1e-8, 0.1
    c = Case(gen(31), n, eight=True, bf16=True, master=True, decay=decay)
    table = gpu_lib.fp8bs_adamw_table([c.dp], [c.dg], [c.dm], [c.dv], master=[c.dw], avg_scales=[c.dms], root_scales=[c.drs],
                                      weight_decay=decay)
    f = lambda x: torch.tensor(x, dtype=torch.float32)  # noqa: E731
    codes, scales = [c.m.clone(), c.v.clone()], [c.ms.clone(), c.rs.clone()]
    for step in range(1000, 1004):
        gpu_lib.fp8bs_adamw_step(table, lr, step, beta1=b1, beta2=b2, eps=eps, seed=seed)
        m, r = (q.view(E4M3).float().view(-1, 128) * s[:, None] for q, s in zip(codes, scales))
        g = c.g.view(-1, 128)
        m = m * f(b1) + g * f(1 - b1)
        r = ((r * r) * f(b2) + (g * g) * f(1 - b2)).double().sqrt().float()   # FP32's on the host is not to nearest
        for i, x in enumerate((m, r)):
            s = x.abs().amax(1) * f(1 / 448)
            q = (x / s[:, None]).clamp(-448, 448)
            if i:
                move = torch.where(q < 2.0 ** -6, 2.0 ** -6, 0.0)
                bits = ((q + move).view(torch.int32).long() + random20(seed, step, 0, n).view(-1, 128)) & ~0xFFFFF
                q = torch.where(x > 0, (bits.to(torch.int32).view(torch.float32) - move).clamp(2.0 ** -9, 448), 0.0)
            codes[i], scales[i] = q.to(E4M3).view(torch.uint8).view(-1), s
    for got, got_s, q, s, label in ((c.dm, c.dms, codes[0], scales[0], "m"), (c.dv, c.drs, codes[1], scales[1], "root")):
        off = ((got.cpu() != q).view(-1, 128).any(1) | (got_s.cpu() != s)).sum()
        assert int(off) <= 8, f"{label}: {int(off)} groups of {n // 128} differ"
