"""Root-mean-square norm with the residual's addition, forward, backward and
straight into FP8 codes, and the router of the experts (softmax, choice of the
best experts, their weights, the balance loss and its gradient): cases of real
use, their plain form in elementary torch operations, their definition in 64
bits, and the calls of this framework's kernels.

Terms.  The residual stream's new value `total` = x + residual is rounded to its
type, and the norm is that of the rounded rows, which the backward pass reads
again.  Blocks of FP8 codes share one scale: 1x128 blocks with an FP32 scale
("block") or 1x32 blocks with an E8M0 byte ("mx"); the transposed codes have
their blocks along the rows.  A router's logits [tokens, experts] give the
probabilities p; token t's choices are its topk largest logits, the lowest
expert first where they are equal; the balance loss is experts * sum over e of
f_e P_e, with f_e the share of the choices that went to expert e and P_e the mean
of p over the tokens; tokens that a mask leaves out (padding) have no choice
(-1) and count nowhere."""
import math

import torch

own = False

FP8 = {"e4m3": (torch.float8_e4m3fn, 448.0, 8), "e5m2": (torch.float8_e5m2, 57344.0, 15)}
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-6


def listed():
    return [
        # the smallest block of the tests and of the latency benchmark, after its residual
        dict(name="rms_fwd_128x512", op="rms", dir="fwd", rows=128, cols=512, ld=512, residual=True, dtype="bf16", wdtype="bf16"),
        # the 405B layer's input
        dict(name="rms_fwd_8192x16384", op="rms", dir="fwd", rows=8192, cols=16384, ld=16384, residual=True, dtype="bf16", wdtype="bf16"),
        # backward through the 8B layer's norm, FP32 weight, with the gradient that comes along the residual stream
        dict(name="rms_bwd_8192x4096", op="rms", dir="bwd", rows=8192, cols=4096, ld=4096, residual=True, dtype="bf16", wdtype="fp32"),
        # an FP32 activation that is a slice of a wider buffer
        dict(name="rms_bwd_1000x4000_fp32", op="rms", dir="bwd", rows=1000, cols=4000, ld=4200, residual=False, dtype="fp32", wdtype="fp32"),
        # a few tokens of the 70B width being generated: the input of one FP8 product
        dict(name="quant_16x8192_mx", op="quant", rows=16, cols=8192, ld=8192, residual=True, dtype="bf16", wdtype="bf16", recipe="mx",
             fmt="e4m3", transposed=False),
        # the 8B layer in training: both orientations, for fprop and wgrad
        dict(name="quant_8192x4096", op="quant", rows=8192, cols=4096, ld=4096, residual=True, dtype="bf16", wdtype="bf16",
             recipe="block", fmt="e4m3", transposed=True),
        # the 405B layer in training
        dict(name="quant_8192x16384", op="quant", rows=8192, cols=16384, ld=16384, residual=True, dtype="bf16", wdtype="fp32",
             recipe="block", fmt="e4m3", transposed=True),
        # a short sequence to eight experts
        dict(name="route_fwd_128x8", op="route", dir="fwd", tokens=128, experts=8, topk=2, dtype="fp32", normalize=True, padded=0.0, given=False),
        # a long batch to many experts, some of it padding
        dict(name="route_fwd_16384x64", op="route", dir="fwd", tokens=16384, experts=64, topk=4, dtype="fp32", normalize=True, padded=0.02,
             given=False),
        # a large batch over a wide choice, BF16 logits (with ties)
        dict(name="route_fwd_65536x256", op="route", dir="fwd", tokens=65536, experts=256, topk=8, dtype="bf16", normalize=False, padded=0.0,
             given=False),
        # the gradient of the long batch's weights and loss
        dict(name="route_bwd_16384x64", op="route", dir="bwd", tokens=16384, experts=64, topk=4, dtype="fp32", normalize=True, padded=0.02,
             given=False),
        # the loss and counts of choices that another rule made, an odd batch
        dict(name="balance_fwd_4095x64", op="route", dir="fwd", tokens=4095, experts=64, topk=8, dtype="fp32", normalize=False, padded=0.0,
             given=True),
    ]


def _log_int(rng, lo, hi, step=1):
    return max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step)


def draw(rng):
    most = max(work(c)["bytes"] for c in listed())
    while True:
        op = rng.choice(["rms", "rms", "quant", "quant", "route", "route", "route"])
        if op == "route":
            experts = _log_int(rng, 2, 512, rng.choice([1, 1, 8]))  # (one expert gets all, whatever the inputs)
            case = dict(op=op, dir=rng.choice(["fwd", "bwd"]), tokens=_log_int(rng, 1, 131072), experts=experts,
                        topk=min(rng.choice([1, 2, 4, 6, 8, 16]), experts), dtype=rng.choice(["fp32", "fp32", "bf16"]),
                        normalize=rng.random() < 0.5, padded=rng.choice([0.0, 0.0, 0.1]), given=rng.random() < 0.25)
            case["given"] = case["given"] and case["topk"] < experts  # (every expert chosen by all: the loss has no gradient)
        else:
            cols = _log_int(rng, 64, 16384) if rng.random() < 0.4 else _log_int(rng, 128, 16384, 128)
            case = dict(op=op, rows=_log_int(rng, 1, 16384), cols=cols, ld=cols + rng.choice([0, 0, 8, 13, 200]),
                        residual=rng.random() < 0.6, dtype=rng.choice(["bf16", "bf16", "fp32"]), wdtype=rng.choice(["bf16", "fp32"]))
            if op == "rms":
                case["dir"] = rng.choice(["fwd", "bwd"])
            else:
                case.update(recipe=rng.choice(["block", "block", "mx"]), fmt=rng.choice(["e4m3", "e4m3", "e5m2"]),
                            transposed=rng.random() < 0.6)
        if work(case)["bytes"] <= most:
            return case


def work(case):
    if case["op"] == "route":
        t, e, k, size = case["tokens"], case["experts"], case["topk"], DTYPES[case["dtype"]].itemsize
        if case["dir"] == "fwd":  # (the slope and the counts: one number per expert each)
            return {"bytes": t * e * size + t * k * (4 if case["given"] else 8) + 8 * e + 4, "flops": t * e * 8}
        return {"bytes": 2 * t * e * size + (0 if case["given"] else t * k * 8) + 4 * e + 4, "flops": t * e * 10}
    e, w = DTYPES[case["dtype"]].itemsize, DTYPES[case["wdtype"]].itemsize
    n = case["rows"] * case["cols"]
    if case["op"] == "quant":
        scales = n * (4 / 128 if case["recipe"] == "block" else 1 / 32)
        out = (n + scales) * (1 + case["transposed"])
        return {"bytes": n * e * (1 + 2 * case["residual"]) + case["cols"] * w + 4 * case["rows"] + out,
                "flops": n * (4 + case["residual"] + 2 * case["transposed"])}
    if case["dir"] == "fwd":
        return {"bytes": n * e * (2 + 2 * case["residual"]) + case["cols"] * w + 4 * case["rows"], "flops": n * (4 + case["residual"])}
    return {"bytes": n * e * (3 + case["residual"]) + 2 * case["cols"] * w + 4 * case["rows"], "flops": n * (9 + case["residual"])}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _mask(case, g):
    """Whole sequences of at most 2048 tokens, whose ends are padding."""
    if not case["padded"]:
        return None
    t = torch.arange(case["tokens"], device="cuda")
    length = min(2048, case["tokens"])
    ends = torch.rand(case["tokens"] // length + 1, generator=g, device="cuda") * 2 * case["padded"] * length
    return t % length < length - ends[t // length]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    s = dict(case)
    if case["op"] == "route":
        t, e, k = case["tokens"], case["experts"], case["topk"]
        s["logits"] = (1.5 * randn(t, e) + 0.5 * randn(1, e)).to(DTYPES[case["dtype"]])
        s["mask"] = _mask(case, g)
        if case["given"]:  # choices of the logits and a bias of each expert's, as a router that balances by it makes them
            biased = s["logits"].float() + 0.5 * randn(1, e)
            s["expert"] = torch.sort(biased, dim=1, descending=True, stable=True).indices[:, :k].to(torch.int32).contiguous()
            if s["mask"] is not None:
                s["expert"][~s["mask"]] = -1
        if case["dir"] == "bwd":
            s["dloss"] = torch.rand((), generator=g, device="cuda") * 0.02
            if not case["given"]:
                s["expert"] = _choose(s["logits"].float(), s["mask"], k)
                s["dweights"] = 1e-2 * randn(t, k)
            s["slope"] = _counts_and_slope(s["expert"], s["mask"], t, e)[1]
        return s
    r, c, ld, dt = case["rows"], case["cols"], case["ld"], DTYPES[case["dtype"]]
    x = randn(r, ld) * torch.exp(0.5 * randn(1, ld))
    x[:, :: 97] *= 20.0  # a few channels far above the others
    s["x"] = x.to(dt)[:, :c]
    s["weight"] = (1.0 + 0.1 * randn(c)).to(DTYPES[case["wdtype"]])
    back = case.get("dir") == "bwd"
    s["residual"] = (2.0 * randn(r, ld)).to(dt)[:, :c] if case["residual"] and not back else None
    if back:  # (x: the rows that the forward pass left)
        s["dy"] = (1e-2 * randn(r, ld)).to(dt)[:, :c]
        s["rstd"] = (s["x"].double().square().mean(1) + EPS).rsqrt().float()
        s["dtotal"] = (1e-2 * randn(r, ld)).to(dt)[:, :c] if case["residual"] else None
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    return _OPS[s["op"], s.get("dir")][own](s)


def _total(s):
    """The rows that are normed, and that they are an output."""
    if s["residual"] is None:
        return s["x"], {}
    total = (s["x"].float() + s["residual"].float()).to(s["x"].dtype)
    return total, {"total": total}


def _rms_plain(s):
    total, out = _total(s)
    h = total.float()
    rstd = 1.0 / torch.sqrt((h * h).mean(1) + EPS)
    return h * rstd[:, None] * s["weight"].float(), {**out, "rstd": rstd}


def _rms_fwd_plain(s):
    y, out = _rms_plain(s)
    return {"y": y.to(s["x"].dtype), **out}


def _rms_fwd_own(s):
    from fp8_scaled_quantization_scale_amd import norm
    y, total, rstd = norm.rms_norm_forward(s["x"], s["weight"], s["residual"], EPS)
    return {"y": y, **({} if s["residual"] is None else {"total": total}), "rstd": rstd}


def _rms_bwd_plain(s):
    h, dy, rstd = s["x"].float(), s["dy"].float(), s["rstd"][:, None]
    n, g = h * rstd, dy * s["weight"].float()
    dx = rstd * (g - n * (g * n).mean(1, keepdim=True))
    if s["dtotal"] is not None:
        dx = dx + s["dtotal"].float()
    return {"dx": dx.to(s["x"].dtype), "dweight": (dy * n).sum(0).to(s["weight"].dtype)}


def _rms_bwd_own(s):
    from fp8_scaled_quantization_scale_amd import norm
    dx, dw = norm.rms_norm_backward(s["dy"], s["x"], s["weight"], s["rstd"], s["dtotal"])
    return {"dx": dx, "dweight": dw}


def _blocks(v, per):
    """v [rows, n] as [rows, ceil(n / per), per], zeros past the end."""
    pad = -v.shape[1] % per
    return (torch.nn.functional.pad(v, (0, pad)) if pad else v).unflatten(1, (-1, per))


def _cast(v, recipe, fmt):
    """FP8 codes [rows, n] of fp32 v and the scales [rows, blocks] that they are multiplied by to stand for v."""
    kind, most, emax = FP8[fmt]
    b = _blocks(v, 128 if recipe == "block" else 32)
    amax = b.abs().amax(2)
    if recipe == "block":
        s = torch.where(amax > 0, torch.full_like(amax, most) / amax, 1.0).clamp(max=torch.finfo(torch.float32).max)
        scales = 1.0 / s
    else:
        mant, exp = torch.frexp(amax)  # amax = mant 2^exp; no element is over the largest, 0.875 2^(emax + 1)
        e = torch.where(amax > 0, (exp - 1 - emax + (mant > 0.875).int()).clamp(-127, 127), 0)
        one = torch.ones_like(amax)
        s, scales = torch.ldexp(one, -e), (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)
    return (b * s[:, :, None]).to(kind).flatten(1)[:, : v.shape[1]], scales


def _quant_plain(s):
    y, out = _rms_plain(s)
    out["codes"], out["scales"] = _cast(y, s["recipe"], s["fmt"])
    if s["transposed"]:
        out["codes_t"], out["scales_t"] = _cast(y.t().contiguous(), s["recipe"], s["fmt"])
    return out


def _quant_own(s):
    import fp8_scaled_quantization_scale_amd as fm
    from fp8_scaled_quantization_scale_amd import norm
    block = s["recipe"] == "block"
    q, total, rstd = norm.rms_norm_quantize(s["x"], fm.BLOCK_1x128 if block else fm.MX_1x32, fm.FMT[s["fmt"]],
                                            fm.ROW_AND_COL if s["transposed"] else fm.ROW, s["weight"], s["residual"], EPS)
    kind, scale = FP8[s["fmt"]][0], torch.float32 if block else torch.float8_e8m0fnu
    out = {**({} if s["residual"] is None else {"total": total}), "rstd": rstd, "codes": q.q_row.view(kind)[:, : s["cols"]],
           "scales": q.s_row.view(scale)}
    if s["transposed"]:
        out.update(codes_t=q.q_col.view(kind)[:, : s["rows"]], scales_t=q.s_col.view(scale))
    return out


def _choose(logits, mask, topk):
    expert = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :topk].to(torch.int32)
    return expert if mask is None else torch.where(mask[:, None], expert, -1)


def _softmax(logits):
    e = torch.exp(logits - logits.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _counts_and_slope(expert, mask, tokens, experts):
    """The choices of each expert, and the derivative of the loss by each p of it (the same for every token)."""
    flat = expert.reshape(-1).long()
    kept = (flat >= 0) & (flat < experts)
    counts = torch.zeros(experts + 1, dtype=torch.int32, device=flat.device)
    counts.index_add_(0, torch.where(kept, flat, experts), kept.int())
    n = torch.full((), float(tokens), device=flat.device) if mask is None else mask.sum().float()
    return counts[:experts], counts[:experts].float() * torch.where(n > 0, experts / (expert.shape[1] * n * n), 0.0)


def _route_fwd_plain(s):
    logits = s["logits"].float()
    p, out = _softmax(logits), {}
    expert = s["expert"] if s["given"] else _choose(logits, s["mask"], s["topk"])
    if not s["given"]:
        w = p.gather(1, expert.clamp(min=0).long())
        if s["normalize"]:
            w = w / w.sum(1, keepdim=True)
        out = {"expert": expert, "weights": torch.where(expert >= 0, w, 0.0)}
    counts, slope = _counts_and_slope(expert, s["mask"], s["tokens"], s["experts"])
    if s["mask"] is not None:
        p = torch.where(s["mask"][:, None], p, 0.0)
    return {**out, "loss": (slope * p.sum(0)).sum(), "counts": counts, "slope": slope}


def _route_fwd_own(s):
    from fp8_scaled_quantization_scale_amd import moe
    if s["given"]:
        loss, counts, slope = moe.balance(s["logits"], s["expert"], s["mask"])
        return {"loss": loss, "counts": counts, "slope": slope}
    r = moe.route(s["logits"], s["topk"], s["normalize"], s["mask"])
    return {"expert": r.expert, "weights": r.weights, "loss": r.loss, "counts": r.counts, "slope": r.slope}


def _route_bwd_plain(s):
    p = _softmax(s["logits"].float())
    dp = (s["dloss"] * s["slope"])[None, :]
    if not s["given"]:
        at = s["expert"].clamp(min=0).long()
        dw = torch.where(s["expert"] >= 0, s["dweights"], 0.0)
        if s["normalize"]:
            w = p.gather(1, at)
            total = w.sum(1, keepdim=True)
            dw = (dw - (dw * w / total).sum(1, keepdim=True)) / total
        dp = dp.expand_as(p).scatter_add(1, at, torch.where(s["expert"] >= 0, dw, 0.0))
    d = p * (dp - (p * dp).sum(1, keepdim=True))
    if s["mask"] is not None:
        d = torch.where(s["mask"][:, None], d, 0.0)
    return {"dlogits": d.to(s["logits"].dtype)}


def _route_bwd_own(s):
    from fp8_scaled_quantization_scale_amd import moe
    if s["given"]:
        return {"dlogits": moe.route_backward(s["logits"], None, None, s["slope"], s["dloss"], mask=s["mask"])}
    return {"dlogits": moe.route_backward(s["logits"], s["expert"], s["dweights"], s["slope"], s["dloss"], s["normalize"], s["mask"])}


_OPS = {("rms", "fwd"): (_rms_fwd_plain, _rms_fwd_own), ("rms", "bwd"): (_rms_bwd_plain, _rms_bwd_own),
        ("quant", None): (_quant_plain, _quant_own), ("route", "fwd"): (_route_fwd_plain, _route_fwd_own),
        ("route", "bwd"): (_route_bwd_plain, _route_bwd_own)}


# ---------------------------------------------------------------------------
# the definition, in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return (_route_exact if s["op"] == "route" else _rms_exact)(s)


def _rms_exact(s):
    n, w = s["cols"], s["weight"].double()
    if s.get("dir") == "bwd":
        dy, r = s["dy"].double(), s["rstd"].double()[:, None]
        h = s["x"].double() * r
        along = (dy * w * h).sum(1, keepdim=True) / n
        dx = (dy * w - along * h) * r
        return {"dx": dx if s["dtotal"] is None else dx + s["dtotal"].double(), "dweight": (dy * h).sum(0)}
    total, out = s["x"].double(), {}
    if s["residual"] is not None:
        out["total"] = total + s["residual"].double()
        total = out["total"].to(s["x"].dtype).double()  # the stream's value is the rounded one
    rstd = ((total ** 2).sum(1) / n + EPS) ** -0.5
    y = total * rstd[:, None] * w
    out["rstd"] = rstd
    if s["op"] == "rms":
        return {"y": y, **out}
    kind, most, _ = FP8[s["fmt"]]
    for name, v in (("", y),) + ((("_t", y.t()),) if s["transposed"] else ()):
        b = _blocks(v, 128 if s["recipe"] == "block" else 32)
        top = b.abs().amax(2)
        inv = torch.where(top > 0, top / most, 1.0)
        if s["recipe"] == "mx":
            inv = 2.0 ** torch.where(top > 0, torch.ceil(torch.log2(inv)), 0.0)
        out["codes" + name] = (b / inv[:, :, None]).clamp(-most, most).to(kind).double().flatten(1)[:, : v.shape[1]]
        out["scales" + name] = inv
    return out


def _route_exact(s):
    logits, t, e, k = s["logits"].double(), s["tokens"], s["experts"], s["topk"]
    real = torch.ones(t, dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"]
    p = torch.softmax(logits, 1) * real[:, None]
    if s["dir"] == "bwd":
        d = p * (s["dloss"].double() * s["slope"].double())
        d = d - p * d.sum(1, keepdim=True)
        if not s["given"]:
            for j in range(k):  # each choice's weight: p by itself, or its share of the chosen
                at = torch.nonzero(s["expert"][:, j] >= 0)[:, 0]
                all_of = s["expert"][at].long()
                pc, dw = p[at].gather(1, all_of), s["dweights"][at, j, None].double()
                w = pc[:, j, None] / (pc.sum(1, keepdim=True) if s["normalize"] else 1.0)
                if s["normalize"]:
                    d[at] = d[at].scatter_add(1, all_of, -dw * w * (pc / pc.sum(1, keepdim=True)))
                else:
                    d[at] = d[at] - dw * w * p[at]
                d[at] = d[at].scatter_add(1, all_of[:, j, None], dw * w)
        return {"dlogits": d}
    if s["given"]:
        expert, out = s["expert"].long(), {}
    else:
        # ties to the lowest: one choice at a time
        left, chosen = logits.clone(), []
        for _ in range(k):
            best = left.amax(1, keepdim=True)
            at = torch.where(left == best, torch.arange(e, device="cuda"), e).amin(1)
            chosen.append(at)
            left[torch.arange(t, device="cuda"), at] = -math.inf
        expert = torch.stack(chosen, 1)
        w = p.gather(1, expert)
        if s["normalize"]:
            w = torch.where(real[:, None], w / w.sum(1, keepdim=True), 0.0)
        out = {"expert": None, "weights": w}
    n = int(real.sum())
    counts = torch.bincount(expert[real].reshape(-1), minlength=e).double()
    share = counts / max(1, n * k)
    return {**out, "loss": e * (share * p.sum(0)).sum() / max(1, n), "counts": None, "slope": e * share / max(1, n)}
