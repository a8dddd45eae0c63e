"""The optimizer step over many steps: weights whose gradient stops, and the states' bits against their rule (adamw_rules)."""

import pytest
import torch

from tests.adamw_rules import States8
from tests.gated_util import E4M3
from tests.linear_util import gen

pytestmark = pytest.mark.gpu


class Weights:
    """n FP32 weights with states in 8 bits, all zero."""

    def __init__(self, lib, n):
        z = lambda k, t=torch.float32: torch.zeros(k, dtype=t, device="cuda")  # noqa: E731
        self.lib, self.p, self.g, self.m, self.r = lib, z(n), z(n), z(n, torch.uint8), z(n, torch.uint8)
        self.ms, self.rs = z(n // 128), z(n // 128)
        self.table = lib.fp8bs_adamw_table([self.p], [self.g], [self.m], [self.r], avg_scales=[self.ms], root_scales=[self.rs])

    def step(self, g, step, beta1, seed=0):
        self.g.copy_(g)
        self.lib.fp8bs_adamw_step(self.table, 1e-3, step, beta1=beta1, beta2=0.95, seed=seed)


@pytest.mark.parametrize("beta1", [0.9, 0.95, 0.99])
def test_weights_without_a_gradient_come_to_rest(gpu_lib, beta1):
    """One column in eight falls silent after 100 steps.  From 448 units m's expected size falls by beta1 a step, so after
    40 / (1 - beta1) more of them it is zero but for one element in 10^13, and the weights stay where they are."""
    n = 4096
    silent = (torch.arange(n, device="cuda") % 8) == 3
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    w, rest = Weights(gpu_lib, n), 100 + int(40 / (1 - beta1))
    for step in range(1, rest + 201):
        grad = torch.randn(n, generator=g, device="cuda") * 1e-3
        w.step(torch.where(silent & (step > 100), 0.0, grad), step, beta1, seed=step)
        if step == rest:
            before = w.p.clone()
    torch.cuda.synchronize()
    assert not (w.m[silent] & 0x7F).any() and torch.equal(w.p[silent], before[silent])
    assert (w.p[~silent] != before[~silent]).all() and torch.isfinite(w.p).all()


@pytest.mark.parametrize("beta1", [0.0, 0.9, 0.9375, 0.95, 0.99])
@pytest.mark.parametrize("small", [1e-5, 1.0])
def test_the_states_follow_their_rule(gpu_lib, beta1, small):
    """Six steps of 2^16 elements, all but one of a group `small` of its size (1e-5: most of them on subnormal codes of m).
    A code may differ where the kernel's quotient, which rounds as the exact one but within 2^-22 of a unit, falls on the
    other side of a rounding boundary: about once in 2^20 codes, and a group with one may differ from then on: 4 of 512."""
    n, steps, seed = 1 << 16, 6, 9
    w, s, g = Weights(gpu_lib, n), States8(n), gen(5)
    size = torch.where(torch.arange(n) % 128 == 0, 1.0, small) * 1e-3
    for step in range(1, steps + 1):
        grad = torch.randn(n, generator=g) * size
        w.step(grad, step, beta1, seed=seed)
        s.step(grad, step, beta1, 0.95, seed=seed)
    torch.cuda.synchronize()
    if small < 1:
        assert (s.m.abs() < 2.0 ** -6).float().mean() > 0.5 and s.m.any()
    for got, scale, want, want_scale, label in ((w.m, w.ms, s.m, s.ms, "m"), (w.r, w.rs, s.r, s.rs, "root")):
        codes = (got.cpu().view(E4M3).float() != want).view(-1, 128).any(1)
        off = int((codes | (scale.cpu() != want_scale)).sum())
        assert off <= 4, f"{label}: {off} groups of {n // 128} differ"


def test_a_first_step_rounds_m_to_nearest(gpu_lib):
    """States that are zero as a whole hold nothing: nothing is left to chance."""
    n = 1 << 14
    w, s = Weights(gpu_lib, n), States8(n, nearest=True)
    grad = torch.randn(n, generator=gen(6)) * torch.where(torch.arange(n) % 128 == 0, 1.0, 1e-5)
    w.step(grad, 1, 0.99)
    s.step(grad, 1, 0.99, 0.95)
    assert torch.equal(w.m.cpu().view(E4M3).float(), s.m)


# ---- large tables pass the caches ---------------------------------------------------------------


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("master", [False, True])
@pytest.mark.parametrize("grad_bf16", [False, True])
def test_large_tables_have_the_bits_of_their_parts(gpu_lib, eight, master, grad_bf16):
    """Tables beyond 128 MiB pass the caches, with new bf16 parameters left in them (no master here: FP32 parameters) or
    not (more than 128 MiB of them): the same bits as a call for each tensor, which has the others' places in the table empty."""
    count, n = 24, (3 << 20) + 77                 # 75 M elements: 302 MB of FP32, 151 MB of bf16
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    randn = lambda k: torch.randn(k, generator=g, device="cuda")  # noqa: E731

    def tensors():
        w = randn(n) * 0.02
        t = dict(p=w.bfloat16() if master else w, g=randn(n) * 1e-3)
        t["g"] = t["g"].bfloat16() if grad_bf16 else t["g"]
        t["master"] = w if master else None
        if eight:
            groups = -(-n // 128)
            t["m"] = torch.randint(0, 256, (n,), generator=g, device="cuda", dtype=torch.uint8)
            t["m"][(t["m"] & 0x7F) == 0x7F] = 0
            t["v"] = torch.randint(0, 0x7F, (n,), generator=g, device="cuda", dtype=torch.uint8)
            t["ms"], t["rs"] = randn(groups).abs() * 1e-6, randn(groups).abs() * 1e-6
        else:
            t["m"], t["v"], t["ms"], t["rs"] = randn(n) * 3e-4, (randn(n) * 1e-3) ** 2, None, None
        return t

    def step(entries):
        of = lambda name: [e[name] for e in entries]  # noqa: E731
        table = gpu_lib.fp8bs_adamw_table(of("p"), of("g"), of("m"), of("v"), master=of("master"), avg_scales=of("ms"),
                                          root_scales=of("rs"), weight_decay=0.1)
        gpu_lib.fp8bs_adamw_step(table, 1e-3, 10, seed=8)

    whole = [tensors() for _ in range(count)]
    parts = [{k: None if x is None else x.clone() for k, x in e.items()} for e in whole]
    step(whole)
    empty = lambda e: {k: None if x is None else x[:0] for k, x in e.items()}  # noqa: E731
    for i, e in enumerate(parts):
        step([empty(o) for o in parts[:i]] + [e])
    torch.cuda.synchronize()
    for i, (a, b) in enumerate(zip(whole, parts)):
        for name in a:
            assert a[name] is None or torch.equal(a[name].view(torch.uint8), b[name].view(torch.uint8)), (i, name)


@pytest.mark.parametrize("eight", [False, True])
def test_large_tables_that_keep_their_parameters(gpu_lib, eight):
    """Beyond 128 MiB in all with fewer than that of bf16 parameters, beside a tensor with a tail: the same bits."""
    n = (8 << 20) + 3
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    entries = []
    for _ in range(2):
        w = torch.randn(n, generator=g, device="cuda")
        e = dict(p=w.bfloat16(), w=w, g=torch.randn(n, generator=g, device="cuda"))
        if eight:
            e.update(m=torch.zeros(n, dtype=torch.uint8, device="cuda"), v=torch.zeros(n, dtype=torch.uint8, device="cuda"),
                     ms=torch.zeros(-(-n // 128), device="cuda"), rs=torch.zeros(-(-n // 128), device="cuda"))
        else:
            e.update(m=torch.zeros(n, device="cuda"), v=torch.zeros(n, device="cuda"), ms=None, rs=None)
        entries.append(e)
    sixteen = lambda e: {k: None if x is None else x.clone() for k, x in e.items()}  # noqa: E731
    parts = [sixteen(e) for e in entries]

    def step(es):
        of = lambda name: [e[name] for e in es]  # noqa: E731
        gpu_lib.fp8bs_adamw_step(gpu_lib.fp8bs_adamw_table(of("p"), of("g"), of("m"), of("v"), master=of("w"),
                                                           avg_scales=of("ms"), root_scales=of("rs")), 1e-3, 1, seed=2)

    # 18 or 12 bytes an element: with FP32 states one tensor alone is beyond 128 MiB, in 8 bits only both together.  The
    # random bits go by the tensor and the element's place, so only FP32 states can be cut, at multiples of a group
    step(entries)
    if eight:
        step([parts[0]])
        empty = {k: None if x is None else x[:0] for k, x in parts[0].items()}
        step([empty, parts[1]])
    else:
        cut = 1 << 20
        for e in parts:
            for at in range(0, n, cut):
                step([{k: None if x is None else x[at:at + cut] for k, x in e.items()}])
    torch.cuda.synchronize()
    for a, b in zip(entries, parts):
        for name in a:
            assert a[name] is None or torch.equal(a[name].view(torch.uint8), b[name].view(torch.uint8)), name
