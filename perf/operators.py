"""Layer norm, expert dispatch and combine, and the grouped scaled FP8 GEMM:
cases of real use, their plain form in elementary torch operations, their
definition in 64 bits, and the calls of this framework's kernels.

Terms.  A router gives each token `topk` experts; the slots (token, choice)
are numbered t * topk + j.  Sorted by expert, slot s sits in row row(s) of a
buffer whose segments, one per expert, start on multiples of 128 rows; the
rows between a segment's last slot and its end are zero, and the rows behind
the last segment belong to nobody.  A slot with an expert outside
[0, experts) is dropped.  Blocks of FP8 codes share one scale: 1x128 blocks
with an FP32 scale ("block") or 1x32 blocks with an E8M0 byte ("mx"); a
weight of the block recipe has 128x128 tiles."""
import itertools
import math
import random

import torch

own = False

ALIGN = 128
FP8 = {"e4m3": (torch.float8_e4m3fn, 448.0, 8), "e5m2": (torch.float8_e5m2, 57344.0, 15)}
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # the smallest block of the tests and of the latency benchmark, before a layer
        dict(name="norm_fwd_128x512", op="norm", dir="fwd", rows=128, cols=512, ld=512, dtype="bf16", wdtype="bf16"),
        # the input of the 405B MLP layer of the benchmark
        dict(name="norm_fwd_8192x16384", op="norm", dir="fwd", rows=8192, cols=16384, ld=16384, dtype="bf16", wdtype="bf16"),
        # the input of the 8B layer, backward in training with FP32 master norms
        dict(name="norm_bwd_8192x4096", op="norm", dir="bwd", rows=8192, cols=4096, ld=4096, dtype="bf16", wdtype="fp32"),
        # an FP32 activation that is a slice of a wider buffer
        dict(name="norm_bwd_1000x4000_fp32", op="norm", dir="bwd", rows=1000, cols=4000, ld=4200, dtype="fp32", wdtype="fp32"),
        # a short sequence to eight experts, both orientations of the codes
        dict(name="dispatch_128x512", op="dispatch", tokens=128, cols=512, experts=8, topk=2, recipe="block", fmt="e4m3",
             weighted=False, dropped=0.0),
        # a long batch to many experts
        dict(name="dispatch_16384x8192", op="dispatch", tokens=16384, cols=8192, experts=64, topk=4, recipe="block", fmt="e4m3",
             weighted=False, dropped=0.02),
        # the way back of the 8B layer's batch
        dict(name="combine_fwd_8192x4096", op="combine", dir="fwd", tokens=8192, cols=4096, experts=8, topk=2, dropped=0.0),
        # its gradient for an odd batch over many experts
        dict(name="combine_bwd_4095x4096", op="combine", dir="bwd", tokens=4095, cols=4096, experts=64, topk=8, dropped=0.02),
        # the tiny block's weight, one for each of eight experts
        dict(name="experts_fprop_128", op="gemm", dir="rows", tokens=128, topk=2, experts=8, n=256, k=512, recipe="block",
             fmt_a="e4m3", fmt_b="e4m3", transposed=False),
        # up-projection of the 8B layer's batch, eight experts
        dict(name="experts_fprop_8192", op="gemm", dir="rows", tokens=8192, topk=2, experts=8, n=14336, k=4096, recipe="block",
             fmt_a="e4m3", fmt_b="e4m3", transposed=False),
        # input gradient through many small experts: E5M2 gradients, MX blocks, the weight's transposed codes
        dict(name="experts_dgrad_4096_mx", op="gemm", dir="rows", tokens=4096, topk=4, experts=64, n=4096, k=2048, recipe="mx",
             fmt_a="e5m2", fmt_b="e4m3", transposed=True),
        # weight gradient of the 8B layer's experts: each contracts over its own rows
        dict(name="experts_wgrad_8192", op="gemm", dir="experts", tokens=8192, topk=2, experts=8, n=14336, k=4096, recipe="block",
             fmt_a="e5m2", fmt_b="e4m3", transposed=False),
    ]


def _log_int(rng, lo, hi, step=1):
    return max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step)


def draw(rng):
    most = max(_cost(c) for c in listed())
    while True:
        op = rng.choice(["norm", "norm", "dispatch", "combine", "gemm", "gemm"])
        if op == "norm":
            cols = _log_int(rng, 64, 16384) if rng.random() < 0.5 else _log_int(rng, 128, 16384, 128)
            case = dict(op=op, dir=rng.choice(["fwd", "bwd"]), rows=_log_int(rng, 1, 16384), cols=cols,
                        ld=cols + rng.choice([0, 0, 8, 13, 200]), dtype=rng.choice(["bf16", "bf16", "fp32"]),
                        wdtype=rng.choice(["bf16", "fp32"]))
        else:
            experts = _log_int(rng, 1, 128)
            topk = min(rng.choice([1, 2, 4, 6, 8]), experts)
            if op == "gemm":
                case = dict(op=op, dir=rng.choice(["rows", "experts"]), tokens=_log_int(rng, 1, 16384), topk=topk, experts=experts,
                            n=_log_int(rng, 16, 14336, rng.choice([8, 128])), k=_log_int(rng, 32, 8192, rng.choice([16, 128])),
                            recipe=rng.choice(["block", "block", "mx"]), fmt_a=rng.choice(["e4m3", "e5m2"]), fmt_b="e4m3",
                            transposed=False)
                if case["dir"] == "rows" and rng.random() < 0.4:  # the weight's transposed codes: whole blocks per expert
                    case.update(transposed=True, n=max(128, case["n"] // 128 * 128), k=max(128, case["k"] // 128 * 128))
            else:
                case = dict(op=op, tokens=_log_int(rng, 1, 32768), cols=_log_int(rng, 16, 8192, rng.choice([16, 128])),
                            experts=experts, topk=topk, dropped=rng.choice([0.0, 0.0, 0.05]))
                if op == "dispatch":
                    case.update(recipe=rng.choice(["block", "block", "mx"]), fmt=rng.choice(["e4m3", "e5m2"]),
                                weighted=rng.random() < 0.5)
                else:
                    case.update(dir=rng.choice(["fwd", "bwd"]))
        if _cost(case) <= most and _memory(case) < 40e9:
            return case


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50)


def _memory(case):  # of the plain form
    if case["op"] != "gemm":
        return 4 * work(case)["bytes"]
    e, n, k = case["experts"], case["n"], case["k"]
    rows = (max(_load(case)[0]) + ALIGN) * e
    return 4.0 * (rows * (2 * k + 2 * n) + 2 * e * n * k)


def work(case):
    if case["op"] == "norm":
        e, w = DTYPES[case["dtype"]].itemsize, DTYPES[case["wdtype"]].itemsize
        r, c = case["rows"], case["cols"]
        if case["dir"] == "fwd":
            return {"bytes": 2 * r * c * e + 2 * c * w + 8 * r, "flops": 8 * r * c}
        return {"bytes": 3 * r * c * e + 3 * c * w + 8 * r, "flops": 14 * r * c}
    t, j = case["tokens"], case["topk"]
    kept = t * j * (1 - case.get("dropped", 0.0))
    if case["op"] == "dispatch":
        c = case["cols"]
        scales = kept * c * 2 * (4 / 128 if case["recipe"] == "block" else 1 / 32)
        return {"bytes": 2 * t * c + 2 * kept * c + scales + t * j * (8 + 4 + 4 + 4 * case["weighted"]), "flops": 4 * kept * c}
    if case["op"] == "combine":
        c = case["cols"]
        if case["dir"] == "fwd":
            return {"bytes": 2 * kept * c + 2 * t * c + 8 * t * j, "flops": 2 * kept * c}
        return {"bytes": 2 * t * c + 4 * kept * c + 12 * t * j, "flops": 3 * kept * c}
    n, k, e = case["n"], case["k"], case["experts"]
    held = min(e, t * j)  # experts that can have rows
    per = 4 / 128 if case["recipe"] == "block" else 1 / 32
    if case["dir"] == "rows":
        return {"bytes": kept * k * (1 + per) + held * n * k * (1 + (per if case["recipe"] == "mx" else 0)) + 2 * kept * n,
                "flops": 2 * kept * n * k}
    return {"bytes": kept * (n + k) * (1 + per) + 2 * e * n * k, "flops": 2 * kept * n * k}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _load(case):
    """How many slots each expert gets, and how many are dropped: a log-normal popularity that is the same for every seed,
    so that the sorted buffers have one size."""
    e, slots = case["experts"], case["tokens"] * case["topk"]
    rng = random.Random(e)
    p = [math.exp(0.7 * rng.gauss(0, 1)) for _ in range(e)]
    dropped = int(slots * case.get("dropped", 0.0))
    ends = [int((slots - dropped) * v / sum(p)) for v in itertools.accumulate(p)]
    ends[-1] = slots - dropped
    return [b - a for a, b in zip([0] + ends, ends)], dropped


def _routing(case, g):
    """int64 experts [tokens, topk], the popular ones more often, -1 where dropped; weights that sum to one."""
    t, e, j = case["tokens"], case["experts"], case["topk"]
    load, dropped = _load(case)
    times = torch.tensor(load + [dropped], device="cuda")
    expert = torch.tensor(list(range(e)) + [-1], device="cuda").repeat_interleave(times, output_size=t * j)
    expert = expert[torch.randperm(t * j, generator=g, device="cuda")].view(t, j)
    return expert, _randn(g, t, j).softmax(1)


def _capacity(tokens, topk, experts):
    slots = tokens * topk
    return (slots + (ALIGN - 1) * min(experts, slots)) // ALIGN * ALIGN


def _sorted(expert, experts):
    """offsets, counts, row_slot, slot_row (int32) of the stable sort by expert."""
    t, j = expert.shape
    flat = expert.reshape(-1).long()
    rows = _capacity(t, j, experts)
    kept = (flat >= 0) & (flat < experts)
    key = torch.where(kept, flat, experts)
    counts = torch.bincount(key, minlength=experts + 1)[: experts + 1]
    counts = counts[:experts]
    padded = (counts + ALIGN - 1) // ALIGN * ALIGN
    offsets = torch.cat([padded.new_zeros(1), padded.cumsum(0)])
    order = torch.sort(key, stable=True).indices
    firsts = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    rank = torch.arange(flat.numel(), device=flat.device) - firsts[key[order]]
    row = torch.where(kept[order], offsets[key[order]] + rank, rows)
    row_slot = torch.full((rows + 1,), -1, dtype=torch.int64, device=flat.device)
    row_slot[row] = torch.where(row < rows, order, -1)
    slot_row = torch.empty_like(flat)
    slot_row[order] = torch.where(row < rows, row, -1)
    i32 = torch.int32
    return offsets.to(i32), counts.to(i32), row_slot[:rows].to(i32), slot_row.view(t, j).to(i32)


def _blocks(x, block):
    """x [..., n] as [..., ceil(n / block), block], zeros past the end."""
    pad = -x.shape[-1] % block
    if pad:
        x = torch.nn.functional.pad(x, (0, pad))
    return x.unflatten(-1, (-1, block))


def _scale(amax, fmt):
    most = FP8[fmt][1]
    s = torch.where(amax > 0, most / amax, 1.0)
    return s.clamp(max=torch.finfo(torch.float32).max)


def _e8m0(amax, fmt):
    """The smallest power of two's exponent under which no element is over the format's largest, plus 127."""
    mant, exp = torch.frexp(amax)  # amax = mant 2^exp, mant in [0.5, 1); the largest is 0.875 2^(emax + 1)
    e = exp - 1 - FP8[fmt][2] + (mant > 0.875).to(exp.dtype)
    return torch.where(amax > 0, e.clamp(-127, 127) + 127, 127).to(torch.uint8)


def _pow2(e):
    return torch.ldexp(torch.ones(e.shape, device=e.device, dtype=torch.float32), e.to(torch.int32))


def _cast(x, recipe, fmt):
    """FP8 codes [.., n] and scales [.., blocks] of fp32 x along its last dimension (the values codes * scales stand for x)."""
    n = x.shape[-1]
    b = _blocks(x, 128 if recipe == "block" else 32)
    amax = b.abs().amax(-1)
    if recipe == "block":
        s = _scale(amax, fmt)
        scales = 1.0 / s
    else:
        scales = _e8m0(amax, fmt)
        s = _pow2(127 - scales.int())
    codes = (b * s.unsqueeze(-1)).to(FP8[fmt][0])
    return codes.flatten(-2)[..., :n], scales


def _cast_tiles(w, fmt):
    """codes [e, n, k] and scales [e, ceil(n/128), ceil(k/128)] of 128x128 tiles."""
    e, n, k = w.shape
    p = torch.nn.functional.pad(w, (0, -k % 128, 0, -n % 128)).unflatten(2, (-1, 128)).unflatten(1, (-1, 128))
    s = _scale(p.abs().amax((2, 4)), fmt)
    codes = (p * s[:, :, None, :, None]).to(FP8[fmt][0]).flatten(3, 4).flatten(1, 2)[:, :n, :k]
    return codes.contiguous(), 1.0 / s


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if case["op"] == "norm":
        r, c, ld, dt, wdt = case["rows"], case["cols"], case["ld"], DTYPES[case["dtype"]], DTYPES[case["wdtype"]]
        x = _randn(g, r, ld) * torch.exp(0.5 * _randn(g, 1, ld)) + 0.3 * _randn(g, r, 1)
        s["x"] = x.to(dt)[:, :c]
        s["weight"] = (1.0 + 0.1 * _randn(g, c)).to(wdt)
        s["bias"] = (0.1 * _randn(g, c)).to(wdt)
        if case["dir"] == "bwd":
            s["dy"] = (1e-2 * _randn(g, r, ld)).to(dt)[:, :c]
            xd = s["x"].double()
            s["mean"] = xd.mean(1).float()
            s["rstd"] = (1.0 / torch.sqrt((xd - xd.mean(1, keepdim=True)).square().mean(1) + 1e-5)).float()
        return s
    expert, weights = _routing(case, g)
    offsets, counts, row_slot, slot_row = _sorted(expert, case["experts"])
    total = int(offsets[-1])
    s.update(expert=expert, weights=weights, total=total)
    if case["op"] == "dispatch":
        x = _randn(g, case["tokens"], case["cols"])
        x[:, :: 97] *= 50.0
        s["x"] = x.bfloat16()
        return s
    s.update(offsets=offsets, counts=counts, row_slot=row_slot, slot_row=slot_row)
    rows = row_slot.numel()
    if case["op"] == "combine":
        s["ys"] = _randn(g, rows, case["cols"]).bfloat16()
        s["ys"][:total] *= (row_slot[:total, None] >= 0)
        if case["dir"] == "bwd":
            s["dy"] = (1e-2 * _randn(g, case["tokens"], case["cols"])).bfloat16()
        return s
    e, n, k, recipe = case["experts"], case["n"], case["k"], case["recipe"]
    held = torch.zeros(rows, dtype=torch.bool, device="cuda")
    held[:total] = row_slot[:total] >= 0
    s["cap"] = int((offsets[1:] - offsets[:-1]).max())
    if case["dir"] == "rows":
        a = _randn(g, rows, k) * held[:, None]
        s["a"], s["s_a"] = _cast(a, recipe, case["fmt_a"])
        s["a"].view(torch.uint8)[total:] = 0x7F  # rows that belong to nobody: NaN codes
        w = 0.02 * _randn(g, e, n, k)
        s["b"], s["s_b"] = _cast_tiles(w, case["fmt_b"]) if recipe == "block" else _cast(w, recipe, case["fmt_b"])
        if case["transposed"]:  # the same matrices, stored [n, e, k]
            s["b"] = s["b"].view(torch.uint8).permute(1, 0, 2).contiguous().permute(1, 0, 2).view(FP8[case["fmt_b"]][0])
            s["s_b"] = s["s_b"].permute(1, 0, 2).contiguous().permute(1, 0, 2)
        return s
    for name, m, fmt in (("a", n, case["fmt_a"]), ("b", k, case["fmt_b"])):
        v = _randn(g, m, rows) * held[None, :]
        s[name], s["s_" + name] = _cast(v, recipe, fmt)
        s[name].view(torch.uint8)[:, total:] = 0x7F
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    return _OPS[s["op"]][own](s)


def _norm_plain(s):
    x, w, b = s["x"].float(), s["weight"].float(), s["bias"].float()
    if s["dir"] == "fwd":
        mean = x.mean(1, keepdim=True)
        d = x - mean
        rstd = 1.0 / torch.sqrt(d.square().mean(1, keepdim=True) + 1e-5)
        return {"y": (d * rstd * w + b).to(s["x"].dtype), "mean": mean[:, 0], "rstd": rstd[:, 0]}
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    h = (x - s["mean"][:, None]) * rstd
    g = dy * w
    dx = rstd * (g - g.mean(1, keepdim=True) - h * (g * h).mean(1, keepdim=True))
    return {"dx": dx.to(s["x"].dtype), "dweight": (dy * h).sum(0).to(s["weight"].dtype), "dbias": dy.sum(0).to(s["weight"].dtype)}


def _norm_own(s):
    from fp8_scaled_quantization_scale_amd import norm
    if s["dir"] == "fwd":
        y, mean, rstd = norm.layer_norm_forward(s["x"], s["weight"], s["bias"], 1e-5)
        return {"y": y, "mean": mean, "rstd": rstd}
    dx, dw, db = norm.layer_norm_backward(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"])
    return {"dx": dx, "dweight": dw, "dbias": db}


def _dispatch_out(s, offsets, counts, row_slot, slot_row, q, s_row, qt, s_col):
    per = 128 if s["recipe"] == "block" else 32
    t = s["total"]
    return {"offsets": offsets, "counts": counts, "row_slot": row_slot, "slot_row": slot_row, "codes": q[:t, : s["cols"]],
            "scales": s_row[:t], "codes_t": qt[:, :t], "scales_t": s_col[:, : t // per]}


def _dispatch_plain(s):
    offsets, counts, row_slot, slot_row = _sorted(s["expert"], s["experts"])
    slot = row_slot.long()
    token = slot.clamp(min=0) // s["topk"]
    x = s["x"].float()[token]
    if s["weighted"]:
        x = x * s["weights"].reshape(-1)[slot.clamp(min=0)][:, None]
    x = torch.where(slot[:, None] >= 0, x, 0.0)
    q, s_row = _cast(x, s["recipe"], s["fmt"])
    qt, s_col = _cast(x.t().contiguous(), s["recipe"], s["fmt"])
    return _dispatch_out(s, offsets, counts, row_slot, slot_row, q, s_row, qt, s_col)


def _dispatch_own(s):
    import fp8_scaled_quantization_scale_amd as fm
    from fp8_scaled_quantization_scale_amd import moe
    plan = moe.sort(s["expert"], s["experts"])
    q = moe.quantize(s["x"], plan, fm.BLOCK_1x128 if s["recipe"] == "block" else fm.MX_1x32, fm.FMT[s["fmt"]], fm.ROW_AND_COL,
                     weights=s["weights"] if s["weighted"] else None)
    t = FP8[s["fmt"]][0]
    return _dispatch_out(s, plan.offsets, plan.counts, plan.row_slot, plan.slot_row, q.q_row.view(t), q.s_row, q.q_col.view(t), q.s_col)


def _combine_plain(s):
    row = s["slot_row"].long()
    kept = row >= 0
    w = torch.where(kept, s["weights"], 0.0)
    if s["dir"] == "fwd":
        y = torch.where(kept[..., None], s["ys"].float()[row.clamp(min=0)], 0.0)
        return {"y": (y * w[..., None]).sum(1).bfloat16()}
    dy, slot = s["dy"].float(), s["row_slot"].long()[: s["total"]]
    at = slot.clamp(min=0)
    g = dy[at // s["topk"]]
    dys = torch.where(slot[:, None] >= 0, g * w.reshape(-1)[at][:, None], 0.0)
    dots = torch.cat([(g * s["ys"][: s["total"]].float()).sum(1), g.new_zeros(1)])
    return {"dys": dys.bfloat16(), "dweights": torch.where(kept, dots[row], 0.0)}


def _combine_own(s):
    from fp8_scaled_quantization_scale_amd import moe
    plan = moe.Plan(s["tokens"], s["topk"], s["experts"], s["row_slot"].numel(), s["offsets"], s["counts"], s["row_slot"], s["slot_row"])
    if s["dir"] == "fwd":
        return {"y": moe.combine(s["ys"], plan, s["weights"])}
    dys, dw = moe.combine_backward(s["dy"], s["ys"], plan, s["weights"])
    return {"dys": dys[: s["total"]], "dweights": dw}


def _values(codes, scales, recipe, tiles=False):
    """fp32 values that codes [.., n] and their scales stand for."""
    v = codes.float()
    if recipe == "mx":
        scales = _pow2(scales.int() - 127)
    if tiles:
        scales = scales.repeat_interleave(128, 1)[:, : v.shape[1]]
    per = 32 if recipe == "mx" else 128
    return v * scales.repeat_interleave(per, -1)[..., : v.shape[-1]]


def _gemm_plain(s):
    # each expert's rows beside the others', as many as the longest has
    off = s["offsets"].long()
    at = off[:-1, None] + torch.arange(s["cap"], device=off.device)
    there = at < off[1:, None]
    at = torch.where(there, at, 0)
    if s["dir"] == "rows":
        a = _values(s["a"], s["s_a"], s["recipe"])[at] if s["total"] else s["a"].new_zeros(at.shape + (s["k"],), dtype=torch.float32)
        a = torch.where(there[..., None], a, 0.0)
        b = _values(s["b"], s["s_b"], s["recipe"], tiles=s["recipe"] == "block")
        c = torch.bmm(a, b.transpose(1, 2).contiguous())
        r = torch.arange(s["total"], device=off.device)
        e = torch.searchsorted(off[1:].contiguous(), r, right=True)
        return {"c": c[e, r - off[e]].bfloat16()}
    a = torch.where(there, _values(s["a"], s["s_a"], s["recipe"])[:, at], 0.0).permute(1, 0, 2).contiguous()
    b = torch.where(there, _values(s["b"], s["s_b"], s["recipe"])[:, at], 0.0).permute(1, 2, 0).contiguous()
    return {"c": torch.bmm(a, b).bfloat16()}


def _gemm_own(s):
    import fp8_scaled_quantization_scale_amd as fm
    from fp8_scaled_quantization_scale_amd import moe
    fa, fb = fm.FMT[s["fmt_a"]], fm.FMT[s["fmt_b"]]
    if s["dir"] == "rows":
        recipe = fm.GEMM_BLOCK_1x128_128x128 if s["recipe"] == "block" else fm.GEMM_MX_1x32
        return {"c": moe.gemm(s["a"], fa, s["s_a"], s["b"], fb, s["s_b"], recipe, s["offsets"])[: s["total"]]}
    recipe = fm.GEMM_BLOCK_1x128_1x128 if s["recipe"] == "block" else fm.GEMM_MX_1x32
    return {"c": moe.gemm_wgrad(s["a"], fa, s["s_a"], s["b"], fb, s["s_b"], recipe, s["offsets"])}


_OPS = {"norm": (_norm_plain, _norm_own), "dispatch": (_dispatch_plain, _dispatch_own),
        "combine": (_combine_plain, _combine_own), "gemm": (_gemm_plain, _gemm_own)}


# ---------------------------------------------------------------------------
# the definition, in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _norm_exact, "dispatch": _dispatch_exact, "combine": _combine_exact, "gemm": _gemm_exact}[case["op"]](s)


def _norm_exact(s):
    x, w, b = s["x"].double(), s["weight"].double(), s["bias"].double()
    n = x.shape[1]
    if s["dir"] == "fwd":
        mu = x.sum(1) / n
        var = ((x - mu[:, None]) ** 2).sum(1) / n
        r = (var + 1e-5) ** -0.5
        return {"y": (x - mu[:, None]) * r[:, None] * w + b, "mean": mu, "rstd": r}
    dy, mu, r = s["dy"].double(), s["mean"].double(), s["rstd"].double()
    h = (x - mu[:, None]) * r[:, None]
    gw = dy * w
    m1, m2 = gw.sum(1) / n, (gw * h).sum(1) / n
    return {"dx": (gw - m1[:, None] - h * m2[:, None]) * r[:, None], "dweight": (dy * h).sum(0), "dbias": dy.sum(0)}


def _segments(expert, experts):
    """For each expert, its slots in order; the segments' starts."""
    flat = expert.reshape(-1).cpu()
    slots = [torch.nonzero(flat == e)[:, 0] for e in range(experts)]
    starts = [0]
    for v in slots:
        starts.append(starts[-1] + -(-v.numel() // ALIGN) * ALIGN)
    return slots, starts


def _dispatch_exact(s):
    slots, starts = _segments(s["expert"], s["experts"])
    x = torch.zeros(starts[-1], s["cols"], dtype=torch.float64, device="cuda")
    for v, at in zip(slots, starts):
        v = v.cuda()
        rows = s["x"][v // s["topk"]].double()
        if s["weighted"]:
            rows = rows * s["weights"].double().reshape(-1)[v][:, None]
        x[at : at + v.numel()] = rows
    kind, most, _ = FP8[s["fmt"]]

    def of(v):
        """The codes' values, each the nearest to its quotient, and what they are multiplied by to stand for v."""
        b = _blocks(v, 128 if s["recipe"] == "block" else 32)
        top = b.abs().amax(-1)
        if s["recipe"] == "block":
            inv = scales = torch.where(top > 0, top / most, 1.0)
        else:  # bytes: whole numbers, held to the plain form's
            inv, scales = 2.0 ** torch.where(top > 0, torch.ceil(torch.log2(top / most)), 0.0), None
        return (b / inv[..., None]).clamp(-most, most).to(kind).double().flatten(-2)[..., : v.shape[-1]], scales

    q, si = of(x)
    qt, st = of(x.t())
    return {"codes": q, "scales": si, "codes_t": qt, "scales_t": st}


def _combine_exact(s):
    row = s["slot_row"].long()
    w, ys = s["weights"].double(), s["ys"]
    if s["dir"] == "fwd":
        y = torch.zeros(s["tokens"], s["cols"], dtype=torch.float64, device="cuda")
        for j in range(s["topk"]):
            t = torch.nonzero(row[:, j] >= 0)[:, 0]
            y[t] += w[t, j, None] * ys[row[t, j]].double()
        return {"y": y}
    dys = torch.zeros(s["total"], s["cols"], dtype=torch.float64, device="cuda")
    dw = torch.zeros(s["tokens"], s["topk"], dtype=torch.float64, device="cuda")
    for j in range(s["topk"]):
        t = torch.nonzero(row[:, j] >= 0)[:, 0]
        d = s["dy"][t].double()
        dys[row[t, j]] = w[t, j, None] * d
        dw[t, j] = (d * ys[row[t, j]].double()).sum(1)
    return {"dys": dys, "dweights": dw}


def _gemm_exact(s):
    def values(codes, scales, rows_per=1):
        per = 128 if s["recipe"] == "block" else 32
        f = scales.double() if s["recipe"] == "block" else 2.0 ** (scales.double() - 127.0)
        i = torch.arange(codes.shape[0], device="cuda") // rows_per
        j = torch.arange(codes.shape[1], device="cuda") // per
        return codes.to(torch.float32).double() * f[i][:, j]

    off = s["offsets"].tolist()
    if s["dir"] == "rows":
        c = torch.zeros(s["total"], s["n"], dtype=torch.float64, device="cuda")
        for e in range(s["experts"]):
            if off[e] < off[e + 1]:
                a = values(s["a"][off[e] : off[e + 1]], s["s_a"][off[e] : off[e + 1]])
                c[off[e] : off[e + 1]] = a @ values(s["b"][e], s["s_b"][e], 128 if s["recipe"] == "block" else 1).t()
        return {"c": c}
    c = torch.zeros(s["experts"], s["n"], s["k"], dtype=torch.float64, device="cuda")
    per = 128 if s["recipe"] == "block" else 32
    for e in range(s["experts"]):
        if off[e] < off[e + 1]:
            lo, hi = off[e], off[e + 1]
            c[e] = values(s["a"][:, lo:hi], s["s_a"][:, lo // per : hi // per]) @ values(s["b"][:, lo:hi], s["s_b"][:, lo // per : hi // per]).t()
    return {"c": c}
