"""Workloads of routing by scores, of the RMS norm with 8-bit rows, and of the 8-bit products, with their plain forms.

Four operators of a routed mixture layer:
  route    scores (sigmoid or softmax), a selection bias, groups of experts, top-k and gates; in training the gates'
           gradient for the logits
  norm     the residual's addition, root-mean-square norm, its rows in float and in 8 bits; in training the gradients
  matmul   rows to 8 bits, and their product with one 8-bit matrix (the shared expert, a dense layer), or with the matrix
           turned: the gradient for the rows
  experts  8-bit rows grouped by expert, each times its expert's 8-bit matrix, or the gradient for the rows

The 8-bit format: E4M3 codes (4 exponent bits, 3 of mantissa, largest 448) with a float32 scale for 128 consecutive values of
a row, or for 128 x 128 values of a matrix: the block's largest magnitude (at least 2^-116) over 448. Rows of codes are
filled up to whole blocks with zeros.
Layer sizes are those of this repository's configurations: hidden size 2048, intermediate size 512, 512 routed experts
and one shared, 10 experts a token; the gate/up matrix of an expert is [1024, 2048], its down matrix [2048, 512].
"""
import math

import torch

own = False

H, I, E, TOPK, B = 2048, 512, 512, 10, 128
LEAST = 2.0 ** -116
F = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # a decode window of 4 tokens: 10 experts out of the best 4 of 8 groups, a bias that balances the load
        {"name": "route window", "op": "route", "T": 4, "E": E, "k": TOPK, "type": "f32", "score": "sigmoid", "bias": True,
         "groups": 8, "keep": 4, "top": 2, "renorm": True, "off": False, "train": False},
        # bfloat16 logits, a number of experts that fits no wave, experts switched off with -inf, softmax scores
        {"name": "route odd", "op": "route", "T": 1000, "E": 100, "k": 8, "type": "bf16", "score": "softmax", "bias": False,
         "groups": 5, "keep": 3, "top": 1, "renorm": False, "off": True, "train": True},
        # a training step over the largest chunk
        {"name": "route training chunk", "op": "route", "T": 8192, "E": E, "k": TOPK, "type": "f32", "score": "sigmoid",
         "bias": True, "groups": 8, "keep": 4, "top": 2, "renorm": True, "off": False, "train": True},
        # one decoded token in front of the router (its rows in bfloat16) and the experts (in 8 bits)
        {"name": "norm one token", "op": "norm", "T": 1, "H": H, "type": "bf16", "weight": "bf16", "residual": True, "out": "both",
         "train": False},
        # a ragged training batch in float32, a hidden size that ends inside a block
        {"name": "norm odd training", "op": "norm", "T": 777, "H": 1000, "type": "f32", "weight": "f32", "residual": True,
         "out": "y", "train": True},
        # the largest prefill chunk, in front of router and experts
        {"name": "norm prefill", "op": "norm", "T": 8192, "H": H, "type": "bf16", "weight": "f32", "residual": True, "out": "both",
         "train": False},
        # the shared expert's gate/up for one decoded token
        {"name": "matmul one token", "op": "matmul", "M": 1, "N": 2 * I, "K": H, "type": "bf16", "grad": False},
        # sizes that fit no tile and end inside a block, float32, the gradient
        {"name": "matmul odd gradient", "op": "matmul", "M": 77, "N": 500, "K": 1000, "type": "f32", "grad": True},
        # the shared expert's gate/up over the largest prefill chunk
        {"name": "matmul prefill", "op": "matmul", "M": 8192, "N": 2 * I, "K": H, "type": "bf16", "grad": False},
        # gate/up of a decode window: 4 tokens pick 10 of 512 experts each, a few of them popular
        {"name": "experts decode", "op": "experts", "T": 4, "E": E, "k": TOPK, "shared": True, "N": 2 * I, "K": H,
         "type": "bf16", "gather": True, "grad": False, "skew": 1.0},
        # gate/up of the largest prefill chunk, experts evenly loaded
        {"name": "experts prefill", "op": "experts", "T": 8192, "E": E, "k": TOPK, "shared": True, "N": 2 * I, "K": H,
         "type": "bf16", "gather": True, "grad": False, "skew": 0.0},
        # the gradient for the tokens through gate/up in a training step, experts unevenly loaded
        {"name": "experts gradient", "op": "experts", "T": 1024, "E": E, "k": TOPK, "shared": True, "N": 2 * I, "K": H,
         "type": "bf16", "gather": True, "grad": True, "skew": 0.3},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def _wide(rng, lo, hi):
    """A matrix's size: as often a multiple of 64 as any number."""
    n = _log(rng, lo, hi)
    return n if rng.random() < 0.5 else max(64, n // 64 * 64)


def draw(rng):
    op = rng.choice(["route", "route", "norm", "norm", "matmul", "matmul", "experts", "experts"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 5, 8, 16])
        n = groups * max(2, _log(rng, 4, 2048) // groups)
        keep = rng.randint(1, groups)
        return {"op": op, "T": min(_log(rng, 1, 8192), 8192 * E // n), "E": n, "k": rng.randint(1, min(keep * n // groups, 12)),
                "type": rng.choice(["f32", "bf16"]), "score": rng.choice(["sigmoid", "softmax"]), "bias": rng.random() < 0.6,
                "groups": groups, "keep": keep, "top": rng.choice([1, 2]), "renorm": rng.random() < 0.6,
                "off": rng.random() < 0.3, "train": rng.random() < 0.5}
    if op == "norm":
        n = _wide(rng, 64, 8192)
        train = rng.random() < 0.5
        return {"op": op, "T": min(_log(rng, 1, 8192), 8192 * H // n // (2 if train else 1)), "H": n, "type": rng.choice(["f32", "bf16"]),
                "weight": rng.choice(["f32", "bf16"]), "residual": rng.random() < 0.6, "out": rng.choice(["y", "fp8", "both"]),
                "train": train}
    if op == "matmul":
        K, N = _wide(rng, 64, 4096), _wide(rng, 64, 4096)
        return {"op": op, "M": min(_log(rng, 1, 8192), 8192 * 2 * I * H // (N * K)), "N": N, "K": K,
                "type": rng.choice(["bf16", "bf16", "f32"]), "grad": rng.random() < 0.4}
    n, k = _log(rng, 8, E), rng.randint(1, 8)
    N, K = _wide(rng, 64, 2048), _wide(rng, 64, 2048)
    return {"op": op, "T": min(_log(rng, 1, 4096), 8192 * TOPK * 2 * I * H // (2 * k * N * K)), "E": n, "k": k,
            "shared": rng.random() < 0.5, "N": N, "K": K, "type": rng.choice(["bf16", "bf16", "f32"]),
            "gather": rng.random() < 0.5, "grad": rng.random() < 0.4, "skew": rng.choice([0.0, 0.3, 0.6])}


# ---- inputs ------------------------------------------------------------------------------------------------------------


def _blocks(v, rows):
    """[..., R, K] as [..., R / rows, rows, K / 128, 128], filled up with zeros (rows is 1 or 128)."""
    v = torch.nn.functional.pad(v.float(), (0, -v.shape[-1] % B, 0, -v.shape[-2] % rows))
    return v.unflatten(-1, (-1, B)).unflatten(-3, (-1, rows))


def _fp8(v, rows=1):
    """Codes [..., R, 128 blocks] and scales [..., R / rows, blocks] of rows v, blocks of `rows` x 128 values."""
    b = _blocks(v, rows)
    scales = b.abs().amax((-3, -1), keepdim=True).clamp_min(LEAST)
    scales = scales / torch.full_like(scales, 448.0)  # by a tensor: a division by a number may be rounded twice
    # in 64 bits: a quotient rounded to 32 first may come to lie on the border between two codes
    m = b.double() / scales.double()
    step = torch.ldexp(torch.ones_like(m), torch.frexp(m).exponent.clamp_min(-5) - 4)
    codes = (torch.round(m / step) * step).clamp(-448, 448).float().to(torch.float8_e4m3fn).flatten(-2).flatten(-3, -2)
    return codes[..., : v.shape[-2], :].contiguous(), scales[..., 0, :, 0]


def _values(codes, scales, K, rows=1):
    """The float32 values [..., R, K] that codes and scales stand for."""
    s = scales.repeat_interleave(B, -1)
    if rows > 1:
        s = s.repeat_interleave(rows, -2)[..., : codes.shape[-2], :]
    return (codes.float() * s)[..., :K]


def _logits(c, g):
    """Router scores: noise, and where `skew` is not 0 a popularity of the experts that falls with their rank."""
    rank = torch.randperm(c["E"], generator=g, device="cuda") + 1
    return torch.randn((c["T"], c["E"]), generator=g, device="cuda") - 1.1 * c.get("skew", 0.0) * rank.float().log()


def _grouping(idx, n, shared):
    T, k = idx.shape
    of = idx.reshape(-1).long()
    if shared:
        of = torch.cat([of, torch.full((T,), n, device=of.device)])
    perm = torch.argsort(of, stable=True)
    slot_of = torch.empty_like(perm)
    slot_of[perm] = torch.arange(len(perm), device=perm.device)
    counts = torch.bincount(of, minlength=n + 1)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    return [t.to(torch.int32) for t in (counts, offsets, perm, slot_of)]


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    s = {"case": c}
    if c["op"] == "route":
        logits = _logits(c, g)
        if c["off"]:
            logits[:, torch.randperm(c["E"], generator=g, device="cuda")[: c["E"] // 10]] = -math.inf
        s["logits"] = logits.to(F[c["type"]])
        s["bias"] = 0.1 * randn(c["E"]) if c["bias"] else None
        s["d_gates"] = randn(c["T"], c["k"])
        s["scale"] = 2.5
    elif c["op"] == "norm":
        t = F[c["type"]]
        s["x"] = (randn(c["T"], c["H"]) * torch.exp(randn(c["T"], 1))).to(t)
        s["residual"] = (randn(c["T"], c["H"]) * 4).to(t) if c["residual"] else None
        s["weight"] = (1 + 0.2 * randn(c["H"])).to(F[c["weight"]])
        s["dy"] = randn(c["T"], c["H"]).to(t)
        s["d_total"] = randn(c["T"], c["H"]).to(t) if c["residual"] else None
        s["eps"] = 1e-6
    else:
        n = 1 if c["op"] == "matmul" else c["E"] + c["shared"]
        s["w_codes"] = torch.empty((n, c["N"], -(-c["K"] // B) * B), dtype=torch.float8_e4m3fn, device="cuda")
        s["w_scales"] = torch.empty((n, -(-c["N"] // B), -(-c["K"] // B)), device="cuda")
        step = max(1, (1 << 26) // (c["N"] * c["K"]))
        for e in range(0, n, step):
            s["w_codes"][e:e + step], s["w_scales"][e:e + step] = _fp8(0.02 * randn(min(step, n - e), c["N"], c["K"]), B)
        rows = c["M"] if c["op"] == "matmul" else c["T"]
        if c["op"] == "matmul":
            s["w_codes"], s["w_scales"] = s["w_codes"][0], s["w_scales"][0]
        else:
            idx = torch.topk(_logits(c, g), c["k"]).indices
            s["counts"], s["offsets"], s["perm"], s["slot_of"] = _grouping(idx, c["E"], c["shared"])
            # what the plain form pads to: the routed experts that have rows, and the most rows that one has
            s["some"] = s["counts"][: c["E"]].nonzero().squeeze(1)
            s["most"] = int(s["counts"][: c["E"]].max())
            if c["grad"] or not c["gather"]:
                rows = c["T"] * (c["k"] + c["shared"])
        x = randn(rows, c["N"] if c["grad"] else c["K"])
        if c["op"] == "matmul":
            s["x"] = x.to(F[c["type"]])
        else:  # the norm, or the gradient's own quantisation, has them in 8 bits
            s["x_codes"], s["x_scales"] = _fp8(x)
    return s


# ---- one pass ----------------------------------------------------------------------------------------------------------


def _plain_route(s):
    c, x = s["case"], s["logits"].float()
    # the order in 64 bits: of two experts whose scores differ in the last place of 32 either might come first
    wide = s["logits"].double()
    if c["score"] == "sigmoid":
        p, choice = 1 / (1 + torch.exp(-x)), 1 / (1 + torch.exp(-wide))
    else:
        top = x.amax(1, keepdim=True)
        ex, choice = torch.exp(x - top), torch.exp(wide - top)
        total = ex.sum(1, keepdim=True)
        p, choice = ex / total, choice / choice.sum(1, keepdim=True)
    if c["bias"]:
        choice = choice + s["bias"].double()
    off = x == -math.inf
    if c["groups"] > 1:
        best = choice.masked_fill(off, -math.inf).unflatten(1, (c["groups"], -1)).sort(dim=-1, descending=True).values[..., : c["top"]]
        there = best != -math.inf
        value = torch.where(there, best, 0).sum(-1).masked_fill(~there.any(-1), -math.inf)
        kept = value.sort(dim=1, descending=True, stable=True).indices[:, : c["keep"]]
        chosen = torch.zeros_like(value, dtype=torch.bool).scatter(1, kept, True).repeat_interleave(c["E"] // c["groups"], 1)
        choice = choice.masked_fill(off, -1e300).masked_fill(~chosen, -math.inf)
    else:
        choice = choice.masked_fill(off, -1e300)
    idx = choice.sort(dim=1, descending=True, stable=True).indices[:, : c["k"]]
    q = p.gather(1, idx)
    total = q.sum(1, keepdim=True)
    if c["renorm"]:
        q = torch.where(total > 0, q / total, 0)
    out = {"idx": idx.to(torch.int32), "gates": s["scale"] * q}
    if c["train"]:
        d = s["scale"] * s["d_gates"]
        if c["renorm"]:
            d = torch.where(total > 0, (d - (d * q).sum(1, keepdim=True)) / total, 0)
        dp = torch.zeros_like(x).scatter(1, idx, d)
        dx = dp * p * (1 - p) if c["score"] == "sigmoid" else p * (dp - (dp * p).sum(1, keepdim=True))
        out["dlogits"] = dx.to(s["logits"].dtype)
    return out


def _plain_norm(s):
    c, t = s["case"], s["x"].dtype
    r, w, out = s["x"].float(), s["weight"].float(), {}
    if c["residual"]:
        r = r + s["residual"].float()
        out["total"] = r.to(t)
    y = r / torch.sqrt(r.square().mean(1, keepdim=True) + s["eps"]) * w
    if c["out"] != "fp8":
        out["y"] = y.to(t)
    if c["out"] != "y":
        out["codes"], out["scales"] = _fp8(y)
    if c["train"]:  # at the rows as they were stored
        r = out["total"].float() if c["residual"] else r
        rms = torch.sqrt(r.square().mean(1, keepdim=True) + s["eps"])
        hat, dy = r / rms, s["dy"].float()
        a = dy * w
        dx = (a - hat * (a * hat).mean(1, keepdim=True)) / rms
        out["dx"] = (dx + s["d_total"].float() if c["residual"] else dx).to(t)
        out["dweight"] = (dy * hat).sum(0)
    return out


def _out(s):
    return F[s["case"]["type"]]


def _plain_matmul(s):
    c = s["case"]
    w = _values(s["w_codes"], s["w_scales"], c["K"], B)
    x = _values(*_fp8(s["x"]), s["x"].shape[1])
    return (x @ (w if c["grad"] else w.t())).to(_out(s))


def _plain_experts(s):
    c = s["case"]
    x = _values(s["x_codes"], s["x_scales"], c["N"] if c["grad"] else c["K"])
    w = _values(s["w_codes"].view(torch.uint8)[s["some"]].view(torch.float8_e4m3fn), s["w_scales"][s["some"]], c["K"], B)
    perm, first, many = s["perm"].long(), s["offsets"][s["some"]].long(), s["counts"][s["some"]].long()
    if c["gather"] and not c["grad"]:
        x = x[torch.where(perm < c["T"] * c["k"], perm // c["k"], perm - c["T"] * c["k"])]
    at = torch.arange(s["most"], device="cuda")
    there = at < many.unsqueeze(1)
    slot = (first.unsqueeze(1) + at).clamp_max(len(perm) - 1)
    y = torch.bmm(x[slot], w if c["grad"] else w.transpose(1, 2))
    full = torch.zeros((len(perm) + 1, y.shape[-1]), device="cuda")
    full[torch.where(there, slot, len(perm))] = y
    y = full[:-1]
    if c["shared"]:  # its group is the last: every token's
        w = _values(s["w_codes"][-1], s["w_scales"][-1], c["K"], B)
        y[-c["T"]:] = x[-c["T"]:] @ (w if c["grad"] else w.t())
    if c["gather"] and c["grad"]:
        of = s["slot_of"].long()
        dx = y[of[: c["T"] * c["k"]]].unflatten(0, (c["T"], c["k"])).sum(1)
        y = dx + y[of[c["T"] * c["k"]:]] if c["shared"] else dx
    return y.to(_out(s))


def run(s):
    c = s["case"]
    if not own:
        return {"route": _plain_route, "norm": _plain_norm, "matmul": _plain_matmul, "experts": _plain_experts}[c["op"]](s)
    import bit_quantized_moe_topk_amd as moe
    if c["op"] == "route":
        idx, gates = moe.route_scores(s["logits"], c["k"], s["bias"], score=c["score"], groups=c["groups"], keep_groups=c["keep"],
                                      group_top=c["top"], renormalize=c["renorm"], scale=s["scale"])
        out = {"idx": idx, "gates": gates}
        if c["train"]:
            out["dlogits"] = moe.route_scores_backward(s["logits"], idx, s["d_gates"], score=c["score"], renormalize=c["renorm"],
                                                       scale=s["scale"])
        return out
    if c["op"] == "norm":
        n = moe.rms_norm(s["x"], s["weight"], s["residual"], eps=s["eps"], rows=c["out"] != "fp8", fp8=c["out"] != "y")
        out = {"total": n.total, "y": n.y}
        if n.fp8 is not None:
            out["codes"], out["scales"] = n.fp8.codes, n.fp8.scales
        if c["train"]:
            out["dx"], out["dweight"] = moe.rms_norm_backward(s["dy"], n.total if c["residual"] else s["x"], s["weight"],
                                                              s["d_total"], eps=s["eps"])
        return out
    w = moe.Fp8(s["w_codes"], s["w_scales"], c["K"], B)
    if c["op"] == "matmul":
        x = moe.fp8_quantize(s["x"])
        return moe.fp8_matmul_backward(x, w, dtype=_out(s)) if c["grad"] else moe.fp8_matmul(x, w, dtype=_out(s))
    x = moe.Fp8(s["x_codes"], s["x_scales"], c["N"] if c["grad"] else c["K"])
    groups = moe.Grouping(s["counts"], s["offsets"], s["perm"], s["slot_of"])
    tokens = c["T"] if c["gather"] else None
    return (moe.fp8_experts_matmul_backward if c["grad"] else moe.fp8_experts_matmul)(x, w, groups, tokens=tokens, dtype=_out(s))


# ---- what a pass cannot do without ---------------------------------------------------------------------------------------


def _touched(c):
    """About how many experts the tokens of a case pick between them."""
    weight = [r ** (-1.1 * c["skew"]) for r in range(1, c["E"] + 1)]
    each = [min(1.0, c["k"] * v / sum(weight)) for v in weight]
    return sum(1 - (1 - p) ** c["T"] for p in each)


def work(case):
    c = case
    size = {"f32": 4, "bf16": 2}[c["type"]]
    if c["op"] == "route":
        n, ids = c["T"] * c["E"], c["T"] * c["k"]
        return {"bytes": n * size * (2 if c["train"] else 1) + 8 * ids + (4 * ids if c["train"] else 0), "flops": n * (20 if c["train"] else 12)}
    if c["op"] == "norm":
        n = c["T"] * c["H"]
        moved = n * size * (1 + 2 * c["residual"] + (c["out"] != "fp8")) + n * (c["out"] != "y") * (1 + 4 / B)
        if c["train"]:
            moved += n * size * (2 + c["residual"])
        return {"bytes": moved + c["H"] * ({"f32": 4, "bf16": 2}[c["weight"]] + 4 * c["train"]), "flops": n * (20 if c["train"] else 8)}
    ins, outs = (c["N"], c["K"]) if c["grad"] else (c["K"], c["N"])
    if c["op"] == "matmul":
        pairs, mats, moved = c["M"], 1, c["M"] * (ins + outs) * size
    else:
        pairs, mats = c["T"] * (c["k"] + c["shared"]), _touched(c) + c["shared"]
        one_in, one_out = c["gather"] and not c["grad"], c["gather"] and c["grad"]
        moved = (c["T"] if one_in else pairs) * ins * (1 + 4 / B) + (c["T"] if one_out else pairs) * outs * size
    return {"bytes": moved + mats * c["N"] * c["K"], "flops": 2 * pairs * c["N"] * c["K"]}


# ---- the definition in 64 bits --------------------------------------------------------------------------------------------


def _value64(codes, scales, K):
    """Sign, four exponent bits, three of mantissa m: (1 + m / 8) 2^(e - 7), or m / 8 * 2^-6 where e is 0; times the scale."""
    n = codes.view(torch.uint8).to(torch.int32)
    e, m = (n >> 3) & 15, (n & 7).double()
    v = torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * torch.exp2((e - 7).double()))
    v = torch.where(n >= 128, -v, v)
    row, col = (torch.arange(n, device=codes.device) for n in v.shape[-2:])
    per = 1 if scales.shape[-2] == v.shape[-2] else B
    return (v * scales.double()[..., row[:, None] // per, col // B])[..., :K]


def _rounded64(v):
    """(E4M3 magnitudes, scales as float32) of rows v [R, K] in 64 bits, each 128 values with a scale; the rows filled up."""
    b = torch.cat([v, v.new_zeros(v.shape[0], -v.shape[1] % B)], 1).view(v.shape[0], -1, B)
    unit = (b.abs().amax(2, keepdim=True).clamp_min(LEAST) / 448).float()
    m = (b / unit.double()).abs()
    grid = _value64(torch.arange(127, dtype=torch.uint8, device=v.device)[None], torch.ones((1, 1), device=v.device), 127)[0]
    mid = (grid[1:] + grid[:-1]) / 2  # past it the upper one; on it the even one
    up = torch.where(torch.arange(126, device=v.device) % 2 == 0, torch.nextafter(mid, mid + 1), mid)
    return (grid[torch.bucketize(m, up, right=True)] * torch.sign(b)).flatten(1), unit.squeeze(2)


def _exact_route(s):
    c = s["case"]
    x = s["logits"].double().requires_grad_()
    p = torch.sigmoid(x) if c["score"] == "sigmoid" else torch.softmax(x, 1)
    order = p.detach() + (s["bias"].double() if c["bias"] else 0)
    off = torch.isneginf(x.detach())
    size = c["E"] // c["groups"]
    if c["groups"] > 1:
        top = torch.topk(torch.where(off, -math.inf, order).view(c["T"], c["groups"], size), min(c["top"], size)).values
        value = torch.where(torch.isneginf(top), 0.0, top).sum(2)
        value = torch.where(torch.isneginf(top[..., 0]), -math.inf, value)
        place = torch.argsort(torch.argsort(value, dim=1, descending=True, stable=True), dim=1)
        lost = (place >= c["keep"]).repeat_interleave(size, 1)
    else:
        lost = torch.zeros_like(off)
    order = torch.where(lost, -math.inf, torch.where(off, -1e300, order))
    idx = torch.argsort(order, dim=1, descending=True, stable=True)[:, : c["k"]]
    q = torch.take_along_dim(p, idx, 1)
    if c["renorm"]:
        q = q / q.sum(1, keepdim=True)
    gates = s["scale"] * q
    out = {"idx": idx.to(torch.int32), "gates": gates.detach()}
    if c["train"]:
        (gates * s["d_gates"].double()).sum().backward()
        out["dlogits"] = x.grad
    return out


def _exact_norm(s):
    c, out = s["case"], {}
    norm = lambda v, w: v * w * torch.rsqrt(v.square().mean(1, keepdim=True) + s["eps"])  # noqa: E731
    r, w = s["x"].double(), s["weight"].double()
    if c["residual"]:
        r = r + s["residual"].double()
        out["total"] = r
    y = norm(r, w)
    if c["out"] != "fp8":
        out["y"] = y
    if c["out"] != "y":
        out["codes"], out["scales"] = _rounded64(y)
    if c["train"]:
        h = r.to(s["x"].dtype).double().requires_grad_()
        w = w.clone().requires_grad_()
        through = (norm(h, w) * s["dy"].double()).sum()
        if c["residual"]:
            through = through + (h * s["d_total"].double()).sum()
        through.backward()
        out["dx"], out["dweight"] = h.grad, w.grad
    return out


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "route":
        return _exact_route(s)
    if c["op"] == "norm":
        return _exact_norm(s)
    if c["op"] == "matmul":
        m, unit = _rounded64(s["x"].double())
        x = (m * unit.double().repeat_interleave(B, 1))[:, : s["x"].shape[1]]
        w = _value64(s["w_codes"], s["w_scales"], c["K"])
        return x @ w if c["grad"] else x @ w.t().contiguous()
    x = _value64(s["x_codes"], s["x_scales"], c["N"] if c["grad"] else c["K"])
    ids = s["perm"].long()
    token = torch.where(ids < c["T"] * c["k"], torch.div(ids, c["k"], rounding_mode="floor"), ids - c["T"] * c["k"])
    y = torch.empty((len(ids), c["K"] if c["grad"] else c["N"]), dtype=torch.float64, device="cuda")
    offsets = s["offsets"].tolist()
    for e in range(s["w_codes"].shape[0]):
        a, b = offsets[e], offsets[e + 1]
        if a < b:
            w = _value64(s["w_codes"][e], s["w_scales"][e], c["K"])
            rows = x[token[a:b]] if c["gather"] and not c["grad"] else x[a:b]
            y[a:b] = rows @ w if c["grad"] else rows @ w.t().contiguous()
    if c["gather"] and c["grad"]:
        return torch.zeros((c["T"], c["K"]), dtype=torch.float64, device="cuda").index_add_(0, token, y)
    return y
