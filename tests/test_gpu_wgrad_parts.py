"""fp8bs_grouped_wgrad_ragged where few tiles over long segments split the rows into parts, with several experts."""

import numpy as np
import pytest
import torch

from tests.linear_util import check
from tests.ragged_rules import CUS, wgrad_parts

pytestmark = pytest.mark.gpu

# (segment lengths, m, n, parts): a segment without rows, segments with fewer slabs than parts (parts without any),
# last slabs of 1 to 63 rows, parts of unequal slabs, several tiles of an expert, rows behind the last segment
CASES = [([9000, 0, 1090], 72, 200, 6), ([2, 5, 1, 14001], 264, 128, 6), ([4133], 256, 136, 8), ([64 * 300 + 63], 8, 8, 32),
         ([0, 6500], 520, 392, 6), ([3333, 3100, 2999], 128, 136, 6)]


def problem(lengths, m, n, tail=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(m + n + len(lengths))
    seg = torch.tensor([0] + list(np.cumsum(lengths)), dtype=torch.int32)
    rows = int(seg[-1]) + tail
    dy = torch.randn((rows, m), generator=g, device="cuda").bfloat16()
    x = torch.randn((rows, n), generator=g, device="cuda").bfloat16()
    if tail:
        dy[-tail:], x[-tail:] = float("nan"), float("inf")
    return seg, dy, x


@pytest.mark.parametrize("lengths,m,n,parts", CASES, ids=lambda v: "-".join(map(str, v)) if isinstance(v, list) else str(v))
def test_parts_join(gpu_lib, lengths, m, n, parts):
    tail = 7 if m % 16 == 8 else 0
    seg, dy, x = problem(lengths, m, n, tail)
    e = len(lengths)
    if torch.cuda.get_device_properties(0).multi_processor_count == CUS:
        assert wgrad_parts(sum(lengths) + tail, e, m, n) == parts
    base = torch.randn((e, m, n), device="cuda")
    base[:, 0, 0] = -0.0
    c = torch.full((e + 1, m, n), float("nan"), device="cuda")
    acc = torch.full((e + 1, m, n), float("nan"), device="cuda")
    acc[:e] = base
    gpu_lib.fp8bs_grouped_wgrad_ragged(dy, x, seg.cuda(), c=c[:e])
    gpu_lib.fp8bs_grouped_wgrad_ragged(dy, x, seg.cuda(), c=acc[:e], accumulate=1)
    torch.cuda.synchronize()
    assert torch.isnan(c[e]).all() and torch.isnan(acc[e]).all()
    for i, length in enumerate(lengths):
        a, b = dy[int(seg[i]):int(seg[i + 1])].double(), x[int(seg[i]):int(seg[i + 1])].double()
        # FP32 sums of exact products: one rounding (of at most twice 2^-24, truncating adders included) per term,
        # and one for each part that is joined
        want, err = (a.t() @ b).cpu(), (2.0 ** -23 * (length + parts + 2) * (a.abs().t() @ b.abs())).cpu()
        check(c[i], want, err, f"expert {i}", bf16=False)
        tot = base[i].double().cpu() + want
        check(acc[i], tot, err + 2.0 ** -24 * (tot.abs() + err), f"expert {i} accumulated", bf16=False)
        if length == 0:
            assert (c[i] == 0).all()
            assert torch.equal(acc[i].view(torch.int32), base[i].view(torch.int32))


def test_one_row_reaches_its_own_expert_only(gpu_lib):
    """Integers, so that every sum is exact: what an expert's neighbours hold cannot hide in a tolerance."""
    lengths, m, n = [9000, 1, 3300, 64], 136, 264
    seg, dy, x = problem(lengths, m, n)
    assert wgrad_parts(sum(lengths), 4, m, n) > 1 or torch.cuda.get_device_properties(0).multi_processor_count != CUS
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    dy = torch.randint(-2, 3, dy.shape, generator=g, device="cuda").bfloat16()
    x = torch.randint(-2, 3, x.shape, generator=g, device="cuda").bfloat16()
    c = gpu_lib.fp8bs_grouped_wgrad_ragged(dy, x, seg.cuda())
    torch.cuda.synchronize()
    for i in range(4):
        cut = slice(int(seg[i]), int(seg[i + 1]))
        assert torch.equal(c[i], (dy[cut].double().t() @ x[cut].double()).float()), i


def test_two_graphs_replayed_at_once(gpu_lib):
    """Each captured call has partial sums of its own, also while the other graph runs."""
    cases = [problem([9000, 0, 1090], 72, 200), problem([3100, 6000, 3500], 72, 200)]
    graphs, outs, want = [], [], []
    for seg, dy, x in cases:
        seg_d = seg.cuda()
        want.append(gpu_lib.fp8bs_grouped_wgrad_ragged(dy, x, seg_d))
        out = torch.empty_like(want[-1])
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            gpu_lib.fp8bs_grouped_wgrad_ragged(dy, x, seg_d, c=out)
        graphs.append((graph, seg_d))
        outs.append(out)
    streams = [torch.cuda.Stream() for _ in cases]
    for i in range(6):
        for out in outs:
            out.fill_(float("nan"))
        torch.cuda.synchronize()
        for _ in range(3):
            for (graph, _), s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    graph.replay()
        torch.cuda.synchronize()
        # the program's own work between the replays
        eager = [gpu_lib.fp8bs_grouped_wgrad_ragged(dy, x, seg_d) for (seg, dy, x), (_, seg_d) in zip(cases, graphs)]
        for out, w, again in zip(outs, want, eager):
            assert torch.equal(out, w) and torch.equal(again, w), i


@pytest.mark.parametrize("rows", [40, 13000])
def test_odd_offsets_and_strides_are_harmless(gpu_lib, rows):
    """Offsets outside the rows are clipped and a backwards segment is empty, split or not; NaN in the columns between
    the matrix and its row stride, and in rows of no segment, reach nothing."""
    m, n = 72, 136
    g = torch.Generator(device="cuda")
    g.manual_seed(rows)
    dy = torch.randint(-2, 3, (rows, m + 16), generator=g, device="cuda").bfloat16()
    x = torch.randint(-2, 3, (rows, n + 8), generator=g, device="cuda").bfloat16()
    dy[:, m:], x[:, n:] = float("nan"), float("inf")
    seg = torch.tensor([-7, 10, 4, rows - 10, 1 << 29], dtype=torch.int32)
    cuts = [slice(0, 10), None, slice(4, rows - 10), slice(rows - 10, rows)]
    c = torch.full((5, m, n), 7.0, device="cuda")
    gpu_lib.fp8bs_grouped_wgrad_ragged(dy[:, :m], x[:, :n], seg.cuda(), c=c[:4])
    torch.cuda.synchronize()
    assert (c[4] == 7.0).all() and (c[1] == 0.0).all()
    for i, cut in enumerate(cuts):
        if cut is not None:
            assert torch.equal(c[i], (dy[cut, :m].double().t() @ x[cut, :n].double()).float()), i
    # a segment that ends before the rows do: what lies behind is not read
    seg = torch.tensor([5, 5, 5, rows - 9, rows - 9], dtype=torch.int32)
    dy[:5], dy[rows - 9:], x[:5], x[rows - 9:] = (float("nan"),) * 4
    gpu_lib.fp8bs_grouped_wgrad_ragged(dy[:, :m], x[:, :n], seg.cuda(), c=c[:4])
    torch.cuda.synchronize()
    assert (c[0] == 0.0).all() and (c[1] == 0.0).all() and (c[3] == 0.0).all()
    cut = slice(5, rows - 9)
    assert torch.equal(c[2], (dy[cut, :m].double().t() @ x[cut, :n].double()).float())
