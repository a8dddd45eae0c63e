"""The cases by which the library's linear-layer and expert operators are timed.

Five operators, as one mixture-of-experts layer with its dense (shared) part uses them:

  linear      y = act(x W^T + bias) + residual from E4M3 codes and their scales, and the same
              epilogue on the activation gradient (the weight read as stored)
  linear_bwd  dz = dy * act'(z) and the bias gradient, the column sums of dz
  route       the expert-major layout of a top-k routing, without padding rows
  experts     the expert matrix products over segments of any length (forward and activation gradient)
  experts_dw  the experts' weight gradients dy_e^T x_e over the same segments, from bf16, in FP32

``run`` computes them in elementary torch operations, or, with ``own`` set, through the library.
Weights and activations come as the library's quantizers leave them: E4M3 codes with one FP32
scale per 1x128 tile of an activation row and per 128x128 block of a weight.
"""

import math

import torch

own = False

GROUP = 128
ACTS = {"none": 0, "relu": 1, "gelu_tanh": 2, "silu": 3}


def listed():
    return [
        # the shared expert's gate projection while serving: four sequences, one token each
        dict(name="linear_decode", kind="linear", m=4, n=4096, k=7168, b_layout=0, act="silu", bias=True,
             residual=False, keep_z=False),
        # a training step's up projection: pre-activations kept for the backward pass
        dict(name="linear_train", kind="linear", m=4096, n=4096, k=7168, b_layout=0, act="gelu_tanh", bias=True,
             residual=False, keep_z=True),
        # the activation gradient of a down projection joining the residual stream's, an odd batch
        dict(name="linear_dgrad_residual", kind="linear", m=1037, n=7168, k=1536, b_layout=1, act="none", bias=False,
             residual=True, keep_z=False),
        # the epilogue's backward pass for a short packed batch
        dict(name="linear_bwd_short", kind="linear_bwd", m=37, n=1536, act="silu"),
        # and for a long one
        dict(name="linear_bwd_long", kind="linear_bwd", m=16384, n=4096, act="gelu_tanh"),
        # routing of eight sequences' next tokens
        dict(name="route_decode", kind="route", tokens=8, topk=8, experts=256, dropped=False),
        # routing of a prompt batch, some pairs dropped
        dict(name="route_prompt", kind="route", tokens=16384, topk=8, experts=256, dropped=True),
        # expert products for eight sequences' next tokens: most touched experts have one row
        dict(name="experts_decode", kind="experts", tokens=8, topk=8, experts=256, n=4096, k=7168, b_layout=0),
        # the expert layer's forward pass over 4096 tokens: 256 experts, top-8
        dict(name="experts_train", kind="experts", tokens=4096, topk=8, experts=256, n=4096, k=7168, b_layout=0),
        # the activation gradient of an expert-parallel rank's 64 experts
        dict(name="experts_dgrad", kind="experts", tokens=1500, topk=8, experts=64, n=7168, k=4096, b_layout=1),
        # weight gradients of a few small experts over a short batch
        dict(name="experts_dw_short", kind="experts_dw", tokens=50, topk=2, experts=8, m=1536, n=512),
        # weight gradients of an expert-parallel rank's 32 experts
        dict(name="experts_dw_train", kind="experts_dw", tokens=2048, topk=8, experts=32, m=4096, n=7168),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["linear", "linear", "linear_bwd", "route", "experts", "experts", "experts_dw"])
    act = rng.choice(sorted(ACTS))
    if kind == "linear":
        return dict(kind=kind, m=_log_int(rng, 1, 4096), n=GROUP * _log_int(rng, 1, 32), k=GROUP * _log_int(rng, 1, 56),
                    b_layout=rng.randrange(2), act=act, bias=rng.random() < 0.6, residual=rng.random() < 0.5,
                    keep_z=rng.random() < 0.4)
    if kind == "linear_bwd":
        return dict(kind=kind, m=_log_int(rng, 1, 16384), n=8 * _log_int(rng, 1, 512), act=act)
    experts = _log_int(rng, 1, {"route": 512, "experts": 64, "experts_dw": 32}[kind])
    topk = rng.randint(1, min(8, experts))
    if kind == "route":
        return dict(kind=kind, tokens=_log_int(rng, 1, 16384), topk=topk, experts=experts, dropped=rng.random() < 0.5)
    tokens = _log_int(rng, 1, 4096)
    if kind == "experts":
        return dict(kind=kind, tokens=tokens, topk=topk, experts=experts, n=GROUP * _log_int(rng, 1, 32),
                    k=GROUP * _log_int(rng, 1, 32), b_layout=rng.randrange(2))
    return dict(kind=kind, tokens=tokens, topk=topk, experts=experts, m=8 * _log_int(rng, 1, 256),
                n=8 * _log_int(rng, 1, 256))


# ---- inputs -------------------------------------------------------------------------------------


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _activation(g, rows, cols, outliers=True):
    """Hidden states: normal values with one percent of the channels much larger."""
    x = _normal(g, rows, cols)
    if outliers:
        x[:, torch.randperm(cols, generator=g, device="cuda")[: max(1, cols // 100)]] *= 20.0
    return x


def _row_tiles(x):
    """E4M3 codes and scales of 1x128 tiles along the columns."""
    t = x.view(x.shape[0], -1, GROUP)
    s = t.abs().amax(2) / 448.0
    q = (t / s.clamp(min=1e-30)[:, :, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return q.view(torch.uint8).view(x.shape), s.contiguous()


def _weight_blocks(g, rows, cols):
    """E4M3 codes and scales of 128x128 blocks of a normal weight of deviation 0.02."""
    w = _normal(g, rows // GROUP, GROUP, cols // GROUP, GROUP) * 0.02
    s = w.abs().amax((1, 3)) / 448.0
    q = (w / s[:, None, :, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return q.view(torch.uint8).view(rows, cols), s.contiguous()


def _topk_ids(g, tokens, topk, experts):
    """Distinct experts for each token, near the balanced loads that a trained router keeps."""
    keys = torch.rand((tokens, experts), generator=g, device="cuda") ** 2
    return keys.topk(topk, 1).indices.to(torch.int32)


def _segments(ids, experts):
    counts = torch.bincount(ids.flatten().long(), minlength=experts)
    return torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)


def prepare(case, seed):
    g, kind, s = _generator(seed), case["kind"], dict(case)
    if kind == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        s["qa"], s["sa"] = _row_tiles(_activation(g, m, k))
        s["qb"], s["sb"] = _weight_blocks(g, n, k) if case["b_layout"] == 0 else _weight_blocks(g, k, n)
        s["bias_v"] = _normal(g, n) if case["bias"] else None
        s["residual_v"] = _normal(g, m, n).bfloat16() if case["residual"] else None
        s["z"] = torch.empty((m, n), dtype=torch.bfloat16, device="cuda") if case["keep_z"] else None
    elif kind == "linear_bwd":
        s["z"] = (_normal(g, case["m"], case["n"]) * 1.5).bfloat16()
        s["dy"] = (_normal(g, case["m"], case["n"]) * 1e-3).bfloat16()
    elif kind == "route":
        ids = _topk_ids(g, case["tokens"], case["topk"], case["experts"])
        if case["dropped"]:
            ids = torch.where(torch.rand(ids.shape, generator=g, device="cuda") < 0.02, -1, ids)
        s["ids"] = ids.to(torch.int32).contiguous()
    else:
        e = case["experts"]
        s["seg"] = _segments(_topk_ids(g, case["tokens"], case["topk"], e), e)
        s["longest"] = int((s["seg"][1:] - s["seg"][:-1]).max())
        rows = case["tokens"] * case["topk"]
        if kind == "experts":
            n, k = case["n"], case["k"]
            s["qa"], s["sa"] = _row_tiles(_activation(g, rows, k))
            shape = (n, k) if case["b_layout"] == 0 else (k, n)
            s["qb"] = torch.empty((e, *shape), dtype=torch.uint8, device="cuda")
            s["sb"] = torch.empty((e, shape[0] // GROUP, shape[1] // GROUP), dtype=torch.float32, device="cuda")
            for i in range(e):
                s["qb"][i], s["sb"][i] = _weight_blocks(g, *shape)
        else:
            s["dy"] = (_normal(g, rows, case["m"]) * 1e-3).bfloat16()
            s["x"] = _activation(g, rows, case["n"]).bfloat16()
    return s


# ---- one pass -----------------------------------------------------------------------------------


def _f32_rows(q, s):
    v = q.view(torch.float8_e4m3fn).float()
    return (v.view(v.shape[0], -1, GROUP) * s[:, :, None]).view(v.shape)


def _f32_blocks(q, s):
    """Stacked weights [..., rows, cols] from codes and block scales."""
    v = q.view(torch.float8_e4m3fn).float()
    blocks = v.view(*v.shape[:-2], s.shape[-2], GROUP, s.shape[-1], GROUP)
    return (blocks * s[..., :, None, :, None]).view(v.shape)


def _act(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z * torch.sigmoid(z)
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu_tanh":
        t = torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z)
    if act == "silu":
        p = torch.sigmoid(z)
        return p + z * p * (1 - p)
    return torch.ones_like(z)


def _places(seg, rows):
    """Each row's expert and place in its segment."""
    seg = seg.long()
    r = torch.arange(rows, device=seg.device)
    e = torch.searchsorted(seg[1:].contiguous(), r, right=True)
    return e, r - seg[e]


def _in_segments(x, e, at, experts, longest):
    """Rows [rows, cols] laid out as [experts, longest, cols], zeros behind each segment."""
    out = x.new_zeros((experts, longest, x.shape[1]))
    out[e, at] = x
    return out


def _plain(s):
    kind = s["kind"]
    if kind == "linear":
        x, w = _f32_rows(s["qa"], s["sa"]), _f32_blocks(s["qb"], s["sb"])
        z = x @ (w.t() if s["b_layout"] == 0 else w)
        if s["bias_v"] is not None:
            z = z + s["bias_v"]
        y = _act(z, s["act"])
        if s["residual_v"] is not None:
            y = y + s["residual_v"].float()
        return {"y": y.bfloat16(), "z": z.bfloat16()} if s["keep_z"] else {"y": y.bfloat16()}
    if kind == "linear_bwd":
        dz = s["dy"].float() * _act_slope(s["z"].float(), s["act"])
        return {"dz": dz.bfloat16(), "dbias": dz.sum(0)}
    if kind == "route":
        flat = s["ids"].flatten().long()
        key = torch.where((flat >= 0) & (flat < s["experts"]), flat, s["experts"])
        counts = torch.bincount(key, minlength=s["experts"] + 1)
        ends = counts[: s["experts"]].cumsum(0)
        order = torch.sort(key, stable=True).indices
        row = torch.empty_like(flat)
        row[order] = torch.arange(flat.numel(), device=flat.device)
        live = key < s["experts"]
        token = torch.where(live[order], order // s["topk"], -1)
        return {"seg": torch.cat([ends.new_zeros(1), ends]).int(),
                "slot_rows": torch.where(live, row, -1).view(s["ids"].shape).int(), "row_token": token.int()}
    experts, longest = s["experts"], s["longest"]
    if kind == "experts":
        x, w = _f32_rows(s["qa"], s["sa"]), _f32_blocks(s["qb"], s["sb"])
        e, at = _places(s["seg"], x.shape[0])
        y = torch.bmm(_in_segments(x, e, at, experts, longest), w.transpose(1, 2) if s["b_layout"] == 0 else w)
        return {"y": y[e, at].bfloat16()}
    dy, x = s["dy"].float(), s["x"].float()
    e, at = _places(s["seg"], x.shape[0])
    return {"dw": torch.bmm(_in_segments(dy, e, at, experts, longest).transpose(1, 2),
                            _in_segments(x, e, at, experts, longest))}


def run(s):
    if not own:
        return _plain(s)
    from fp8_fine_grained_act_amd import lib

    kind = s["kind"]
    if kind == "linear":
        y = lib.fp8bs_gemm_epilogue(s["qa"], s["sa"], s["qb"], s["sb"], b_layout=s["b_layout"], bias=s["bias_v"],
                                    act=ACTS[s["act"]], residual=s["residual_v"], z=s["z"])
        return {"y": y, "z": s["z"]} if s["keep_z"] else {"y": y}
    if kind == "linear_bwd":
        dz, dbias = lib.fp8bs_epilogue_backward(s["dy"], s["z"], act=ACTS[s["act"]])
        return {"dz": dz, "dbias": dbias}
    if kind == "route":
        seg, slot_rows, row_token = lib.fp8bs_moe_route_ragged(s["ids"], s["experts"])
        return {"seg": seg, "slot_rows": slot_rows, "row_token": row_token}
    if kind == "experts":
        return {"y": lib.fp8bs_grouped_gemm_ragged(s["qa"], s["sa"], s["seg"], s["qb"], s["sb"],
                                                   b_layout=s["b_layout"])}
    return {"dw": lib.fp8bs_grouped_wgrad_ragged(s["dy"], s["x"], s["seg"])}


# ---- what a pass cannot do without --------------------------------------------------------------


def _touched(case):
    """Expected number of experts that own a row."""
    return case["experts"] * (1.0 - (1.0 - case["topk"] / case["experts"]) ** case["tokens"])


def work(case):
    kind = case["kind"]
    if kind == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        outs = 1 + bool(case["residual"]) + bool(case["keep_z"])
        return {"bytes": m * k * (1 + 4 / GROUP) + n * k * (1 + 4 / GROUP ** 2) + 2 * m * n * outs + 4 * n * bool(case["bias"]),
                "flops": 2 * m * n * k}
    if kind == "linear_bwd":
        reads = 1 if case["act"] == "none" else 2
        return {"bytes": 2 * case["m"] * case["n"] * (reads + 1) + 4 * case["n"], "flops": 10 * case["m"] * case["n"]}
    if kind == "route":
        return {"bytes": 12 * case["tokens"] * case["topk"] + 4 * (case["experts"] + 1), "flops": 0}
    rows = case["tokens"] * case["topk"]
    if kind == "experts":
        n, k = case["n"], case["k"]
        return {"bytes": rows * k * (1 + 4 / GROUP) + _touched(case) * n * k * (1 + 4 / GROUP ** 2) + 2 * rows * n,
                "flops": 2 * rows * n * k}
    m, n = case["m"], case["n"]
    return {"bytes": 2 * rows * (m + n) + 4 * case["experts"] * m * n, "flops": 2 * rows * m * n}


# ---- the definition, in 64 bits -----------------------------------------------------------------


def _f64(q):
    """E4M3 codes (1 sign, 4 exponent, 3 fraction bits, bias 7) as doubles, by the format's definition."""
    code = torch.arange(256, device=q.device)
    exponent, fraction = (code >> 3) & 15, (code & 7).double()
    value = torch.where(exponent == 0, fraction * 2.0 ** -9, (8 + fraction) * 2.0 ** (exponent.double() - 10))
    return torch.where(code >= 128, -value, value)[q.long()]


def _product64(qa, sa, qb, sb, b_layout):
    """sum over 128-long blocks kb of sa[:, kb] * sb[block] * (codes' partial product), in 64 bits."""
    n = qb.shape[0] if b_layout == 0 else qb.shape[1]
    c = torch.zeros((qa.shape[0], n), dtype=torch.float64, device=qa.device)
    for kb in range(qa.shape[1] // GROUP):
        cut = slice(kb * GROUP, (kb + 1) * GROUP)
        part = _f64(qa[:, cut]) @ (_f64(qb[:, cut]).t() if b_layout == 0 else _f64(qb[cut]))
        sn = (sb[:, kb] if b_layout == 0 else sb[kb]).double().repeat_interleave(GROUP)
        c += sa[:, kb].double()[:, None] * sn[None, :] * part
    return c


def exact(case, seed):
    s, kind = prepare(case, seed), case["kind"]
    if kind == "linear":
        z = _product64(s["qa"], s["sa"], s["qb"], s["sb"], s["b_layout"])
        if s["bias_v"] is not None:
            z += s["bias_v"].double()
        if s["act"] == "relu":
            y = torch.where(z > 0, z, torch.zeros_like(z))
        elif s["act"] == "gelu_tanh":  # (1 + tanh u) / 2 = 1 / (1 + exp(-2u))
            y = z / (1 + torch.exp(-2 * (2 / math.pi) ** 0.5 * (z + 0.044715 * z ** 3)))
        elif s["act"] == "silu":
            y = z / (1 + torch.exp(-z))
        else:
            y = z.clone()
        if s["residual_v"] is not None:
            y += s["residual_v"].double()
        return {"y": y, "z": z} if s["keep_z"] else {"y": y}
    if kind == "linear_bwd":
        z, dy = s["z"].double(), s["dy"].double()
        if s["act"] == "relu":
            slope = torch.where(z > 0, 1.0, 0.0)
        elif s["act"] == "gelu_tanh":  # d/dz of z / (1 + exp(-v))
            v = 2 * (2 / math.pi) ** 0.5 * (z + 0.044715 * z ** 3)
            dv = 2 * (2 / math.pi) ** 0.5 * (1 + 3 * 0.044715 * z ** 2)
            slope = 1 / (1 + torch.exp(-v)) + z * dv / (2 + torch.exp(v) + torch.exp(-v))
        elif s["act"] == "silu":
            slope = 1 / (1 + torch.exp(-z)) + z / (2 + torch.exp(z) + torch.exp(-z))
        else:
            slope = torch.ones_like(z)
        return {"dz": dy * slope, "dbias": (dy * slope).sum(0)}
    if kind == "route":
        ids = s["ids"].cpu().tolist()
        runs = [[] for _ in range(case["experts"])]
        for t, slots in enumerate(ids):
            for j, e in enumerate(slots):
                if 0 <= e < case["experts"]:
                    runs[e].append((t, j))
        seg, rows, token = [0], [[-1] * case["topk"] for _ in ids], []
        for run_e in runs:
            for t, j in run_e:
                rows[t][j] = len(token)
                token.append(t)
            seg.append(len(token))
        token += [-1] * (len(ids) * case["topk"] - len(token))
        return {"seg": torch.tensor(seg, dtype=torch.int32), "slot_rows": torch.tensor(rows, dtype=torch.int32),
                "row_token": torch.tensor(token, dtype=torch.int32)}
    seg = s["seg"].tolist()
    if kind == "experts":
        y = torch.zeros((seg[-1], case["n"]), dtype=torch.float64, device="cuda")
        for e in range(case["experts"]):
            cut = slice(seg[e], seg[e + 1])
            if seg[e + 1] > seg[e]:
                y[cut] = _product64(s["qa"][cut], s["sa"][cut], s["qb"][e], s["sb"][e], s["b_layout"])
        return {"y": y}
    dw = torch.zeros((case["experts"], case["m"], case["n"]), dtype=torch.float64, device="cuda")
    for e in range(case["experts"]):
        cut = slice(seg[e], seg[e + 1])
        dw[e] = s["dy"][cut].double().t() @ s["x"][cut].double()
    return {"dw": dw}
