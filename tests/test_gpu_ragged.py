"""Routing without padding rows, and the expert products and weight gradients over ragged segments, on the GPU."""

import numpy as np
import pytest
import torch

from tests.linear_util import blocks, check, gen, normal, product64, row_tiles

pytestmark = pytest.mark.gpu


# ---- routing ------------------------------------------------------------------------------------


def route_plain(ids, experts):
    runs = [[] for _ in range(experts)]
    for t, slots in enumerate(ids.tolist()):
        for j, e in enumerate(slots):
            if 0 <= e < experts:
                runs[e].append((t, j))
    seg, slot, tok = [0], -np.ones(ids.shape, np.int32), []
    for r in runs:
        for t, j in r:
            slot[t, j] = len(tok)
            tok.append(t)
        seg.append(len(tok))
    return np.array(seg, np.int32), slot, np.array(tok, np.int32)


@pytest.mark.parametrize("tokens,topk,experts", [(0, 2, 4), (1, 1, 1), (1, 8, 256), (8, 8, 256), (65, 3, 7), (64, 1, 64),
                                                 (1000, 8, 512), (1025, 6, 160), (5000, 4, 33), (16384, 8, 256)])
def test_route_ragged(gpu_lib, tokens, topk, experts):
    rng = np.random.default_rng(tokens + topk + experts)
    for kind in ("spread", "dropped", "one expert"):
        ids = rng.integers(0, experts, (tokens, topk)).astype(np.int32)
        if kind == "dropped":
            ids[rng.random(ids.shape) < 0.3] = -1
            ids[rng.random(ids.shape) < 0.1] = experts
        if kind == "one expert":
            ids[:] = experts - 1
        cap = tokens * topk + 37
        seg, slot, tok = gpu_lib.fp8bs_moe_route_ragged(torch.from_numpy(ids).cuda(), experts, rows_cap=cap)
        torch.cuda.synchronize()
        rs, rl, rt = route_plain(ids, experts)
        assert np.array_equal(seg.cpu().numpy(), rs), kind
        assert np.array_equal(slot.cpu().numpy(), rl), kind
        got = tok.cpu().numpy()
        assert np.array_equal(got[:len(rt)], rt) and (got[len(rt):] == -1).all(), kind


# ---- expert products ----------------------------------------------------------------------------


def seg_of(lengths, first=0):
    return torch.tensor([first] + list(first + np.cumsum(lengths)), dtype=torch.int32)


LENGTHS = [[1], [0], [5], [16], [17, 0, 1], [0, 0, 64, 0], [65, 1, 0, 15, 16], [128, 129, 127, 1], [300, 2, 0, 193],
           [1] * 20, [3, 0] * 70, [200, 190, 210, 180]]


@pytest.mark.parametrize("b_layout", [0, 1])
@pytest.mark.parametrize("lengths", LENGTHS, ids=lambda v: "-".join(map(str, v[:5])) + f"x{len(v)}")
def test_grouped_products(gpu_lib, lengths, b_layout):
    n, k = (256, 384) if len(lengths) > 10 else (384, 640)
    e = len(lengths)
    g = gen(sum(lengths) + e + b_layout)
    lead, tail = (3, 5) if e % 2 else (0, 0)                     # rows before the first and behind the last segment
    rows = lead + sum(lengths) + tail
    seg = seg_of(lengths, lead)
    qa, sa = row_tiles(normal(g, rows, k))
    qb, sb = blocks(normal(g, *((e, n, k) if b_layout == 0 else (e, k, n))) * 0.05)
    c = torch.full((rows, n + 8), 9.0, dtype=torch.bfloat16, device="cuda")
    # what lies outside the segments must not matter: NaN codes and scales there
    qa_d, sa_d = qa.clone(), sa.clone()
    for cut in (slice(0, lead), slice(rows - tail, rows)):
        qa_d[cut] = 0x7F
        sa_d[cut] = float("nan")
    gpu_lib.fp8bs_grouped_gemm_ragged(qa_d.cuda(), sa_d.cuda(), seg.cuda(), qb.cuda(), sb.cuda(), b_layout=b_layout,
                                      c=c[:, :n])
    torch.cuda.synchronize()
    assert (c[:, n:] == 9.0).all() and (c[:lead] == 9.0).all() and (c[rows - tail:] == 9.0).all()
    for i in range(e):
        cut = slice(int(seg[i]), int(seg[i + 1]))
        if cut.start == cut.stop:
            continue
        y, err = product64(qa[cut], sa[cut], qb[i], sb[i], b_layout)
        check(c[cut, :n], y, err, f"expert {i} of {lengths[:6]}")


@pytest.mark.parametrize("b_layout", [0, 1])
def test_long_contraction_and_wide_outputs(gpu_lib, b_layout):
    for lengths, n, k in (([2, 1, 0, 3], 128, 7168), ([40, 9, 33], 2048, 1024), ([150, 260, 90], 1152, 2048)):
        e, g = len(lengths), gen(n + k)
        seg = seg_of(lengths)
        qa, sa = row_tiles(normal(g, int(seg[-1]), k))
        qb, sb = blocks(normal(g, *((e, n, k) if b_layout == 0 else (e, k, n))) * 0.05)
        c = gpu_lib.fp8bs_grouped_gemm_ragged(qa.cuda(), sa.cuda(), seg.cuda(), qb.cuda(), sb.cuda(), b_layout=b_layout)
        torch.cuda.synchronize()
        for i in range(e):
            cut = slice(int(seg[i]), int(seg[i + 1]))
            if cut.start < cut.stop:
                y, err = product64(qa[cut], sa[cut], qb[i], sb[i], b_layout)
                check(c[cut], y, err, f"expert {i}")


def test_odd_offsets_are_harmless(gpu_lib):
    """Offsets outside the rows are clipped and a backwards segment is empty: nothing outside c is written."""
    n, k, rows = 256, 256, 40
    g = gen(1)
    qa, sa = row_tiles(normal(g, rows, k))
    qb, sb = blocks(normal(g, 4, n, k) * 0.05)
    big = torch.full((rows + 64, n), 9.0, dtype=torch.bfloat16, device="cuda")
    seg = torch.tensor([-7, 10, 4, 30, 1 << 29], dtype=torch.int32)      # experts 0: 0..10, 1: none, 2: 4..30, 3: 30..40
    gpu_lib.fp8bs_grouped_gemm_ragged(qa.cuda(), sa.cuda(), seg.cuda(), qb.cuda(), sb.cuda(), c=big[:rows])
    torch.cuda.synchronize()
    assert (big[rows:] == 9.0).all()
    y, err = product64(qa[:4], sa[:4], qb[0], sb[0], 0)
    check(big[:4], y, err, "clipped below")
    y, err = product64(qa[30:], sa[30:], qb[3], sb[3], 0)
    check(big[30:rows], y, err, "clipped above")


def test_grouped_products_equal_the_padded_layout(gpu_lib):
    """The segments of fp8bs_moe_route are a special case: every routed row as fp8bs_grouped_gemm gives it."""
    g = gen(77)
    e, n, k = 6, 512, 1024
    counts = [130, 0, 5, 256, 1, 70]
    padded = [(c + 127) // 128 * 128 for c in counts]
    seg = seg_of(padded)
    rows = int(seg[-1])
    qa, sa = row_tiles(normal(g, rows, k))
    qb, sb = blocks(normal(g, e, n, k) * 0.05)
    dev = [t.cuda() for t in (qa, sa, seg, qb, sb)]
    a = gpu_lib.fp8bs_grouped_gemm(*dev)
    b = gpu_lib.fp8bs_grouped_gemm_ragged(*dev)
    torch.cuda.synchronize()
    y = a.double().cpu()
    x = qa.view(torch.float8_e4m3fn).double().abs() * sa.double().repeat_interleave(128, 1)
    mag = torch.zeros_like(y)
    for i in range(e):
        w = qb[i].view(torch.float8_e4m3fn).double().abs() * sb[i].double().repeat_interleave(128, 0).repeat_interleave(128, 1)
        cut = slice(int(seg[i]), int(seg[i + 1]))
        mag[cut] = x[cut] @ w.t()
    check(b, y, 2 * (2.0 ** -10 + (k // 128 + 2) * 2.0 ** -24) * mag + 2.0 ** -8 * y.abs(), "padded layout")


# ---- weight gradients ---------------------------------------------------------------------------


@pytest.mark.parametrize("lengths", LENGTHS + [[1000, 3]], ids=lambda v: "-".join(map(str, v[:5])) + f"x{len(v)}")
@pytest.mark.parametrize("m,n", [(8, 8), (128, 136), (200, 264)])
def test_wgrad(gpu_lib, lengths, m, n):
    e, g = len(lengths), gen(sum(lengths) + m + n)
    lead, tail = (3, 5) if e % 2 else (0, 0)
    rows = lead + sum(lengths) + tail
    seg = seg_of(lengths, lead)
    dy, x = normal(g, rows, m + 8).bfloat16(), normal(g, rows, n + 16).bfloat16()
    for t in (dy, x):                                            # what lies outside the segments must not matter
        t[:lead] = float("nan")
        t[rows - tail:] = float("inf")
    dyd, xd = dy.cuda()[:, :m], x.cuda()[:, :n]
    want = torch.zeros((e, m, n), dtype=torch.float64)
    mag = torch.zeros_like(want)
    for i in range(e):
        a, b = dy[int(seg[i]):int(seg[i + 1]), :m].double(), x[int(seg[i]):int(seg[i + 1]), :n].double()
        want[i], mag[i] = a.t() @ b, a.abs().t() @ b.abs()
    # FP32 sums of exact products: one rounding (of at most twice 2^-24, truncating adders included) per term
    err = 2.0 ** -23 * (max(lengths) + 2) * mag
    c = torch.full((e + 1, m, n), float("nan"), device="cuda")
    gpu_lib.fp8bs_grouped_wgrad_ragged(dyd, xd, seg.cuda(), c=c[:e])
    torch.cuda.synchronize()
    check(c[:e], want, err, "overwritten", bf16=False)
    assert torch.isnan(c[e]).all()
    norm = float((c[:e].double().cpu() - want).norm() / want.norm()) if float(want.norm()) else 0.0
    assert norm <= 1e-6, f"normwise {norm:.2e}"
    base = normal(g, e, m, n)
    acc = base.cuda()
    gpu_lib.fp8bs_grouped_wgrad_ragged(dyd, xd, seg.cuda(), c=acc, accumulate=1)
    torch.cuda.synchronize()
    tot = base.double() + want
    check(acc, tot, err + 2.0 ** -24 * (tot.abs() + err), "accumulated", bf16=False)


def test_wgrad_no_rows(gpu_lib):
    seg = torch.zeros(4, dtype=torch.int32, device="cuda")
    dy, x = torch.empty((0, 16), dtype=torch.bfloat16, device="cuda"), torch.empty((0, 24), dtype=torch.bfloat16, device="cuda")
    c = torch.full((3, 16, 24), 2.0, device="cuda")
    gpu_lib.fp8bs_grouped_wgrad_ragged(dy, x, seg, c=c, accumulate=1)
    torch.cuda.synchronize()
    assert (c == 2.0).all()
    gpu_lib.fp8bs_grouped_wgrad_ragged(dy, x, seg, c=c)
    torch.cuda.synchronize()
    assert (c == 0.0).all()


def test_wgrad_larger_tiles(gpu_lib):
    """Shapes over several tiles and many slabs, against float64 on the device."""
    g = gen(4)
    for lengths, m, n in (([700, 0, 1300], 640, 1152), ([64, 2000], 1024, 512), ([4096], 256, 384)):
        e, seg = len(lengths), seg_of(lengths)
        dy, x = (normal(g, int(seg[-1]), m) * 1e-3).bfloat16().cuda(), normal(g, int(seg[-1]), n).bfloat16().cuda()
        c = gpu_lib.fp8bs_grouped_wgrad_ragged(dy, x, seg.cuda())
        for i in range(e):
            a, b = dy[int(seg[i]):int(seg[i + 1])].double(), x[int(seg[i]):int(seg[i + 1])].double()
            w, mag = a.t() @ b, a.abs().t() @ b.abs()
            check(c[i], w.cpu(), (2.0 ** -23 * (lengths[i] + 2) * mag).cpu(), f"{lengths[i]} rows", bf16=False)


def test_streams_and_graph(gpu_lib):
    """The chain on another stream, and captured and replayed with other routings in the same buffers."""
    g = gen(21)
    tokens, topk, e, h, f = 40, 3, 10, 256, 384
    ids = torch.randint(0, e, (tokens, topk), generator=g, dtype=torch.int32).cuda()
    x = normal(g, tokens, h).bfloat16().cuda()
    wq, ws = (t.cuda() for t in blocks(normal(g, e, f, h) * 0.05))
    gates = torch.rand((tokens, topk), generator=g).cuda()
    rows = tokens * topk

    def bufs():
        return dict(seg=torch.empty(e + 1, dtype=torch.int32, device="cuda"),
                    slot=torch.empty((tokens, topk), dtype=torch.int32, device="cuda"),
                    tok=torch.empty(rows, dtype=torch.int32, device="cuda"),
                    q=torch.empty((rows, h), dtype=torch.uint8, device="cuda"),
                    s=torch.empty((rows, h // 128), device="cuda"),
                    y=torch.empty((rows, f), dtype=torch.bfloat16, device="cuda"),
                    dw=torch.empty((e, f, h), device="cuda"),
                    xr=torch.randn((rows, h), device="cuda").bfloat16(),
                    out=torch.empty((tokens, f), dtype=torch.bfloat16, device="cuda"))

    def chain(b, stream=None):
        gpu_lib.fp8bs_moe_route_ragged(ids, e, seg_offsets=b["seg"], slot_rows=b["slot"], row_token=b["tok"], stream=stream)
        gpu_lib.fp8bs_moe_permute_quantize(x, b["slot"], b["seg"], b["tok"], q=b["q"], scales=b["s"], stream=stream)
        gpu_lib.fp8bs_grouped_gemm_ragged(b["q"], b["s"], b["seg"], wq, ws, c=b["y"], stream=stream)
        gpu_lib.fp8bs_moe_combine(b["y"], b["slot"], gates, out=b["out"], stream=stream)
        gpu_lib.fp8bs_grouped_wgrad_ragged(b["y"], b["xr"], b["seg"], c=b["dw"], stream=stream)

    b0, b1 = bufs(), bufs()
    b1["xr"].copy_(b0["xr"])
    chain(b0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    chain(b1, s)
    torch.cuda.synchronize()
    for name in b0:
        assert torch.equal(b0[name].view(torch.uint8), b1[name].view(torch.uint8)), name
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain(b1)
    for i in range(4):
        new = torch.randint(-1, e, (tokens, topk), generator=g, dtype=torch.int32)
        if i == 2:
            new[:] = -1                                          # nothing routed at all
        ids.copy_(new)
        for b in (b0, b1):
            b["y"].zero_()
        chain(b0)
        graph.replay()
        torch.cuda.synchronize()
        total = int(b0["seg"][-1])
        for name in ("seg", "slot", "tok", "out", "y", "dw"):
            u, v = b0[name], b1[name]
            assert torch.equal(u.view(torch.uint8), v.view(torch.uint8)), (i, name)
        assert torch.equal(b0["q"][:total], b1["q"][:total])


@pytest.mark.parametrize("b_layout", [0, 1])
@pytest.mark.parametrize("low,high,n", [(0, 8, 2048), (40, 80, 1024), (100, 150, 1024), (190, 256, 1024), (0, 600, 1024)])
def test_every_tile_height(gpu_lib, low, high, n, b_layout):
    """64 experts with few to many rows each: every tile height that the call chooses among."""
    rng = np.random.default_rng(low + high)
    lengths = [int(v) for v in rng.integers(low, high + 1, 64)]
    lengths[5], lengths[63] = 0, high
    k, e, g = 384, 64, gen(high)
    seg = seg_of(lengths)
    qa, sa = row_tiles(normal(g, int(seg[-1]), k))
    qb, sb = blocks(normal(g, *((e, n, k) if b_layout == 0 else (e, k, n))) * 0.05)
    dev = [t.cuda() for t in (qa, sa, qb, sb)]
    c = gpu_lib.fp8bs_grouped_gemm_ragged(dev[0], dev[1], seg.cuda(), dev[2], dev[3], b_layout=b_layout)
    torch.cuda.synchronize()
    for i in range(e):
        cut = slice(int(seg[i]), int(seg[i + 1]))
        if cut.start < cut.stop:
            y, err = product64(dev[0][cut], dev[1][cut], dev[2][i], dev[3][i], b_layout)
            check(c[cut], y.cpu(), err.cpu(), f"expert {i}, {lengths[i]} rows")


def test_large_routing_in_a_graph(gpu_lib):
    """The three launches of a large routing, captured and replayed on other ids in the same buffers."""
    g = gen(31)
    tokens, topk, e = 3000, 5, 100
    ids = torch.randint(-1, e + 1, (tokens, topk), generator=g, dtype=torch.int32).cuda()
    out = gpu_lib.fp8bs_moe_route_ragged(ids, e)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gpu_lib.fp8bs_moe_route_ragged(ids, e, seg_offsets=out[0], slot_rows=out[1], row_token=out[2])
    for _ in range(3):
        ids.copy_(torch.randint(-1, e + 1, (tokens, topk), generator=g, dtype=torch.int32))
        want = gpu_lib.fp8bs_moe_route_ragged(ids, e)
        for t in out:
            t.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b)
        rs, rl, rt = route_plain(ids.cpu().numpy(), e)
        assert np.array_equal(out[0].cpu().numpy(), rs) and np.array_equal(out[1].cpu().numpy(), rl)
        assert np.array_equal(out[2].cpu().numpy()[:len(rt)], rt)


def test_wgrad_many_tiles(gpu_lib):
    """More tiles than workgroups, so that tiles follow one another: short, long and empty segments in turn."""
    g = gen(77)
    lengths = [1, 300, 0, 64, 65, 0, 0, 130, 5, 200] * 8
    e, m, n = len(lengths), 520, 1032
    seg = seg_of(lengths)
    dy, x = normal(g, int(seg[-1]), m).bfloat16().cuda(), normal(g, int(seg[-1]), n).bfloat16().cuda()
    base = torch.randn((e, m, n), device="cuda")
    c = torch.full((e, m, n), float("nan"), device="cuda")
    gpu_lib.fp8bs_grouped_wgrad_ragged(dy, x, seg.cuda(), c=c)
    acc = gpu_lib.fp8bs_grouped_wgrad_ragged(dy, x, seg.cuda(), c=base.clone(), accumulate=1)
    torch.cuda.synchronize()
    for i in range(e):
        a, b = dy[int(seg[i]):int(seg[i + 1])].double(), x[int(seg[i]):int(seg[i + 1])].double()
        want, err = (a.t() @ b).cpu(), (2.0 ** -23 * (lengths[i] + 2) * (a.abs().t() @ b.abs())).cpu()
        check(c[i], want, err, f"expert {i}", bf16=False)
        tot = base[i].double().cpu() + want
        check(acc[i], tot, err + 2.0 ** -24 * (tot.abs() + err), f"expert {i} accumulated", bf16=False)


@pytest.mark.parametrize("lengths,m,n", [([4096], 256, 136), ([3000, 0, 1090], 72, 200), ([1024, 5, 1, 4097], 264, 128)])
def test_wgrad_split_over_rows(gpu_lib, lengths, m, n):
    """Few tiles over long segments: the rows are split and the parts joined, the same bits every time."""
    g, e = gen(m + n), len(lengths)
    seg = seg_of(lengths)
    dy, x = normal(g, int(seg[-1]), m).bfloat16().cuda(), normal(g, int(seg[-1]), n).bfloat16().cuda()
    base = torch.randn((e, m, n), device="cuda")
    base[:, 0, 0] = -0.0
    c = gpu_lib.fp8bs_grouped_wgrad_ragged(dy, x, seg.cuda())
    acc = gpu_lib.fp8bs_grouped_wgrad_ragged(dy, x, seg.cuda(), c=base.clone(), accumulate=1)
    torch.cuda.synchronize()
    for i in range(e):
        a, b = dy[int(seg[i]):int(seg[i + 1])].double(), x[int(seg[i]):int(seg[i + 1])].double()
        want, err = (a.t() @ b).cpu(), (2.0 ** -23 * (lengths[i] + 2) * (a.abs().t() @ b.abs())).cpu()
        check(c[i], want, err, f"expert {i}", bf16=False)
        tot = base[i].double().cpu() + want
        check(acc[i], tot, err + 2.0 ** -24 * (tot.abs() + err), f"expert {i} accumulated", bf16=False)
        if lengths[i] == 0:
            assert torch.equal(acc[i].view(torch.int32), base[i].view(torch.int32))
    # on another stream, and captured and replayed on other rows
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    d = gpu_lib.fp8bs_grouped_wgrad_ragged(dy, x, seg.cuda(), stream=s)
    torch.cuda.synchronize()
    assert torch.equal(c, d)
    seg_d, out = seg.cuda(), torch.empty_like(c)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gpu_lib.fp8bs_grouped_wgrad_ragged(dy, x, seg_d, c=out)
    for i in range(4):
        dy.copy_(dy.roll(i + 1, 0))
        want = gpu_lib.fp8bs_grouped_wgrad_ragged(dy, x, seg_d)
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), i
