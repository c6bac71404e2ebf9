"""Workloads of the microscaled 4-bit expert products and of the router's balance loss, with their plain forms.

Four operators of a routed mixture layer:
  quantize   rows to microscaled 4-bit blocks and back to the values they stand for
  matmul     rows times one microscaled matrix (the shared expert, a dense layer), or its gradient for the rows
  experts    rows grouped by expert, each times its expert's microscaled matrix, or the gradient for the rows
  balance    per-expert counts, balance loss and z loss of a router, and their gradient for the logits

The block format: 32 consecutive values share one scale byte s that stands for 2^(s - 127) (255: the block is NaN);
a value is a sign and one of 0, 0.5, 1, 1.5, 2, 3, 4, 6, two to a byte, the first in the low half.
Layer sizes are those of this repository's configurations: hidden size 2048, intermediate size 512, 512 routed experts
and one shared, 10 experts a token; the gate/up matrix of an expert is [1024, 2048], its down matrix [2048, 512].
"""
import math

import torch

own = False

H, I, E, TOPK = 2048, 512, 512, 10
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
F = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # the activations of 16 decode streams of 4 tokens, before a product of two 4-bit operands
        {"name": "quantize 64 rows", "op": "quantize", "rows": 64, "K": H, "type": "bf16"},
        # weights at load time: gate and up of 64 experts
        {"name": "quantize 64 experts", "op": "quantize", "rows": 64 * 2 * I, "K": H, "type": "f32"},
        # the shared expert's gate/up for one decoded token
        {"name": "matmul one token", "op": "matmul", "M": 1, "N": 2 * I, "K": H, "type": "bf16", "grad": False},
        # sizes that fit no tile: a ragged batch, and a last block that is not full
        {"name": "matmul odd f32", "op": "matmul", "M": 77, "N": 500, "K": 1000, "type": "f32", "grad": False},
        # the shared expert's gate/up over a prefill chunk whose activations are 4-bit too
        {"name": "matmul prefill mx4", "op": "matmul", "M": 8192, "N": 2 * I, "K": H, "type": "mx4", "grad": False},
        # gate/up of a decode window: 4 tokens pick 10 of 512 experts each, a few of them popular
        {"name": "experts decode", "op": "experts", "T": 4, "E": E, "k": TOPK, "shared": True, "N": 2 * I, "K": H,
         "type": "bf16", "gather": True, "grad": False, "skew": 1.0},
        # down of a batched decode step in float32: rows that lie in the groups' order
        {"name": "experts batched f32", "op": "experts", "T": 64, "E": E, "k": TOPK, "shared": True, "N": H, "K": I,
         "type": "f32", "gather": False, "grad": False, "skew": 1.0},
        # gate/up of the largest prefill chunk, experts evenly loaded
        {"name": "experts prefill", "op": "experts", "T": 8192, "E": E, "k": TOPK, "shared": True, "N": 2 * I, "K": H,
         "type": "bf16", "gather": True, "grad": False, "skew": 0.0},
        # the gradient for the tokens through gate/up in a training step, experts unevenly loaded
        {"name": "experts gradient", "op": "experts", "T": 1024, "E": E, "k": TOPK, "shared": True, "N": 2 * I, "K": H,
         "type": "bf16", "gather": True, "grad": True, "skew": 0.3},
        # the smallest training batch
        {"name": "balance 64 tokens", "op": "balance", "T": 64, "E": E, "k": TOPK, "type": "f32", "masked": False, "skew": 1.0},
        # a padded batch, bfloat16 logits, an expert count that fits no wave, experts switched off with -inf
        {"name": "balance padded odd", "op": "balance", "T": 1000, "E": 100, "k": 8, "type": "bf16", "masked": True, "skew": 0.5},
        # a training step over a full chunk
        {"name": "balance 8192 tokens", "op": "balance", "T": 8192, "E": E, "k": TOPK, "type": "f32", "masked": False, "skew": 1.0},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def _wide(rng, lo, hi):
    """A matrix's size: as often a multiple of 64 as any number."""
    n = _log(rng, lo, hi)
    return n if rng.random() < 0.5 else max(64, n // 64 * 64)


def draw(rng):
    op = rng.choice(["quantize", "matmul", "matmul", "experts", "experts", "balance"])
    if op == "quantize":
        K = _wide(rng, 32, 4096)
        return {"op": op, "rows": min(_log(rng, 1, 65536), 64 * 2 * I * H // K), "K": K, "type": rng.choice(["f32", "bf16"])}
    if op == "matmul":
        K, N, kind = _wide(rng, 64, 4096), _wide(rng, 64, 4096), rng.choice(["bf16", "bf16", "f32", "mx4"])
        return {"op": op, "M": min(_log(rng, 1, 8192), 8192 * 2 * I * H // (N * K)), "N": N, "K": K, "type": kind,
                "grad": kind != "mx4" and rng.random() < 0.4}
    if op == "experts":
        n, k = _log(rng, 8, E), rng.randint(1, 8)
        N, K, kind = _wide(rng, 64, 2048), _wide(rng, 64, 2048), rng.choice(["bf16", "bf16", "f32", "mx4"])
        return {"op": op, "T": min(_log(rng, 1, 4096), 8192 * TOPK * 2 * I * H // (2 * k * N * K)), "E": n, "k": k, "shared": rng.random() < 0.5, "N": N, "K": K,
                "type": kind, "gather": rng.random() < 0.5, "grad": kind != "mx4" and rng.random() < 0.4,
                "skew": rng.choice([0.0, 0.3, 0.6])}
    n = _log(rng, 4, 2048)
    return {"op": op, "T": min(_log(rng, 1, 8192), 8192 * E // n), "E": n, "k": rng.randint(1, min(n, 12)),
            "type": rng.choice(["f32", "bf16"]), "masked": rng.random() < 0.4, "skew": rng.choice([0.0, 0.5, 1.0])}


# ---- inputs ------------------------------------------------------------------------------------------------------------


def _blocks(v):
    """[..., K] as float32 blocks [..., ceil(K / 32), 32], the last one filled up with zeros."""
    v = torch.nn.functional.pad(v.float(), (0, -v.shape[-1] % 32))
    return v.unflatten(-1, (-1, 32))


def _quantized(v):
    """Codes (a number 0 .. 15 a value) and scale bytes of the blocks of `v`: the scale is the power of two that puts the
    block's largest value in [4, 8), values go to the nearest of the grid, halves to the even one, past 6 to 6."""
    b = _blocks(v)
    top = b.abs().amax(-1, keepdim=True)
    e = torch.where(top > 0, torch.frexp(top).exponent - 3, torch.full_like(top, -127, dtype=torch.int32)).clamp_min(-127)
    m = torch.ldexp(torch.ldexp(b.abs(), -(e // 2)), e // 2 - e)
    code = ((m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5)).to(torch.uint8)
    return code + 8 * torch.signbit(b).to(torch.uint8), (e + 127).squeeze(-1).to(torch.uint8)


def _packed(code):
    return (code[..., 0::2] + 16 * code[..., 1::2]).flatten(-2)


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


def _logits(c, g):
    """Router scores: noise, and where `skew` is not 0 a popularity of the experts that falls with their rank."""
    rank = torch.randperm(c["E"], generator=g, device="cuda") + 1
    return torch.randn((c["T"], c["E"]), generator=g, device="cuda") - 1.1 * c["skew"] * rank.float().log()


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    s = {"case": c}
    if c["op"] == "quantize":
        s["x"] = (randn(c["rows"], c["K"]) * torch.exp(randn(c["rows"], 1))).to(F[c["type"]])
    elif c["op"] == "balance":
        logits = _logits(c, g)
        if c["masked"]:
            logits[:, torch.randperm(c["E"], generator=g, device="cuda")[: (c["E"] - c["k"]) // 8]] = -math.inf
            s["mask"] = torch.arange(c["T"], device="cuda") % 128 < 100
        s["logits"] = logits.to(F[c["type"]])
        s["idx"] = torch.topk(s["logits"].float(), c["k"]).indices.to(torch.int32)
        s["d_losses"] = torch.tensor([1e-2, 1e-3], device="cuda") * (1 + torch.rand(2, generator=g, device="cuda"))
    else:
        n = 1 if c["op"] == "matmul" else c["E"] + c["shared"]
        blocks = -(-c["K"] // 32)
        s["w_codes"] = torch.empty((n, c["N"], 16 * blocks), dtype=torch.uint8, device="cuda")
        s["w_scales"] = torch.empty((n, c["N"], blocks), dtype=torch.uint8, device="cuda")
        step = max(1, (1 << 26) // (c["N"] * c["K"]))
        for e in range(0, n, step):
            code, s["w_scales"][e:e + step] = _quantized(0.02 * randn(min(step, n - e), c["N"], c["K"]))
            s["w_codes"][e:e + step] = _packed(code)
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
        if c["type"] == "mx4":
            code, s["x_scales"] = _quantized(x)
            s["x_codes"] = _packed(code)
        else:
            s["x"] = x.to(F[c["type"]])
    return s


# ---- one pass ----------------------------------------------------------------------------------------------------------


def _values(codes, scales, K):
    """The float32 values that packed codes [..., 16 B] and scales [..., B] stand for, [..., K]."""
    table = torch.tensor(GRID + tuple(-v for v in GRID), device=codes.device)
    v = table[torch.stack([codes & 15, codes >> 4], -1).long()].unflatten(-2, (-1, 16)).flatten(-2)
    return (v * torch.exp2(scales.float() - 127).unsqueeze(-1)).flatten(-2)[..., :K]


def _plain_quantize(s):
    code, scales = _quantized(s["x"])
    return _values(_packed(code), scales, s["case"]["K"])


def _plain_x(s):
    return _values(s["x_codes"], s["x_scales"], s["case"]["K"]) if s["case"]["type"] == "mx4" else s["x"].float()


def _out(s):
    return torch.float32 if s["case"]["type"] == "f32" else torch.bfloat16


def _plain_matmul(s):
    w = _values(s["w_codes"], s["w_scales"], s["case"]["K"])
    return (_plain_x(s) @ (w if s["case"]["grad"] else w.t())).to(_out(s))


def _plain_experts(s):
    c = s["case"]
    x, w = _plain_x(s), _values(s["w_codes"][s["some"]], s["w_scales"][s["some"]], c["K"])
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
        w = _values(s["w_codes"][-1], s["w_scales"][-1], c["K"])
        y[-c["T"]:] = x[-c["T"]:] @ (w if c["grad"] else w.t())
    if c["gather"] and c["grad"]:
        of = s["slot_of"].long()
        dx = y[of[: c["T"] * c["k"]]].unflatten(0, (c["T"], c["k"])).sum(1)
        y = dx + y[of[c["T"] * c["k"]:]] if c["shared"] else dx
    return y.to(_out(s))


def _plain_balance(s):
    c = s["case"]
    x = s["logits"].float()
    keep = s["mask"].float() if c["masked"] else torch.ones(c["T"], device="cuda")
    n = keep.sum()
    counts = torch.zeros(c["E"], device="cuda").index_add(0, s["idx"].flatten().long(), keep.repeat_interleave(c["k"]))
    top = x.amax(1, keepdim=True)
    ex = torch.exp(x - top)
    total = ex.sum(1, keepdim=True)
    p = ex / total
    lse = (top + torch.log(total)).squeeze(1)
    share = counts / (n * c["k"])
    balance = c["E"] * (share * (p * keep.unsqueeze(1)).sum(0) / n).sum()
    z = (keep * lse.square()).sum() / n
    inner = share - (p * share).sum(1, keepdim=True)
    d = p * (s["d_losses"][0] * c["E"] / n * inner + s["d_losses"][1] * 2 / n * lse.unsqueeze(1)) * keep.unsqueeze(1)
    return torch.stack([balance, z]), counts.to(torch.int32), d.to(s["logits"].dtype)


def run(s):
    c = s["case"]
    if not own:
        return {"quantize": _plain_quantize, "matmul": _plain_matmul, "experts": _plain_experts, "balance": _plain_balance}[c["op"]](s)
    import bit_quantized_moe_topk_amd as moe
    if c["op"] == "quantize":
        return moe.mx4_dequantize(moe.mx4_quantize(s["x"]))
    if c["op"] == "balance":
        out = moe.balance_loss(s["logits"], s["idx"], s.get("mask"))
        return out.losses, out.counts, moe.balance_loss_backward(s["logits"], out, s["d_losses"], s.get("mask"))
    w = moe.Mx4(s["w_codes"], s["w_scales"], c["K"])
    x = moe.Mx4(s["x_codes"], s["x_scales"], c["K"]) if c["type"] == "mx4" else s["x"]
    if c["op"] == "matmul":
        return moe.mx4_matmul_backward(x, w) if c["grad"] else moe.mx4_matmul(x, w)
    groups = moe.Grouping(s["counts"], s["offsets"], s["perm"], s["slot_of"])
    tokens = c["T"] if c["gather"] else None
    if c["grad"]:
        return moe.mx4_experts_matmul_backward(x, w, groups, tokens=tokens)
    return moe.mx4_experts_matmul(x, w, groups, tokens=tokens)


# ---- what a pass cannot do without ---------------------------------------------------------------------------------------


def _touched(c):
    """About how many experts the tokens of a case pick between them."""
    weight = [r ** (-1.1 * c["skew"]) for r in range(1, c["E"] + 1)]
    each = [min(1.0, c["k"] * v / sum(weight)) for v in weight]
    return sum(1 - (1 - p) ** c["T"] for p in each)


def work(case):
    c = case
    size = {"f32": 4, "bf16": 2, "mx4": 17 / 32}[c["type"]]
    if c["op"] == "quantize":
        n = c["rows"] * c["K"]
        return {"bytes": n * (size + 17 / 32 + 4), "flops": 4 * n}
    if c["op"] == "balance":
        n = c["T"] * c["E"]
        return {"bytes": 2 * n * size + 4 * c["T"] * c["k"], "flops": 12 * n}
    out = 4 if c["type"] == "f32" else 2
    if c["op"] == "matmul":
        rows, pairs, mats = c["M"], c["M"], 1
        ins, outs = (c["N"], c["K"]) if c["grad"] else (c["K"], c["N"])
        moved = rows * (ins * size + outs * out)
    else:
        pairs = c["T"] * (c["k"] + c["shared"])
        mats = _touched(c) + c["shared"]
        ins, outs = (c["N"], c["K"]) if c["grad"] else (c["K"], c["N"])
        one_in, one_out = c["gather"] and not c["grad"], c["gather"] and c["grad"]
        moved = (c["T"] if one_in else pairs) * ins * size + (c["T"] if one_out else pairs) * outs * out
    return {"bytes": moved + mats * c["N"] * c["K"] * 17 / 32, "flops": 2 * pairs * c["N"] * c["K"]}


# ---- the definition in 64 bits --------------------------------------------------------------------------------------------


def _value64(codes, scales, K):
    """Sign, two exponent bits and a mantissa bit: (1 + m / 2) 2^(e - 1), or m / 2 where e is 0; times 2^(s - 127)."""
    lo, hi = codes.to(torch.int16) & 15, codes.to(torch.int16) >> 4
    n = torch.stack([lo, hi], -1).flatten(-2)
    e, m = (n >> 1) & 3, (n & 1).double()
    v = torch.where(e == 0, m / 2, (1 + m / 2) * torch.exp2((e - 1).double()))
    v = torch.where(n >= 8, -v, v)
    return (v * torch.exp2(scales.double() - 127).repeat_interleave(32, -1))[..., :K]


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "quantize":
        x = s["x"].double()
        x = torch.cat([x, x.new_zeros(c["rows"], -c["K"] % 32)], 1).view(c["rows"], -1, 32)
        unit = torch.exp2(torch.floor(torch.log2(x.abs().amax(2, keepdim=True).clamp_min(2.0 ** -125))) - 2)
        m = x.abs() / unit
        step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0)).double()
        q = (torch.round(m / step) * step).clamp_max(6.0) * torch.sign(x) * unit
        return q.flatten(1)[:, : c["K"]]
    if c["op"] == "balance":
        x = s["logits"].double().requires_grad_()
        keep = s["mask"] if c["masked"] else torch.ones(c["T"], dtype=torch.bool, device="cuda")
        kept, idx = x[keep], s["idx"][keep].long()
        counts = torch.bincount(idx.flatten(), minlength=c["E"])
        p = torch.softmax(kept, 1)
        losses = torch.stack([c["E"] * (counts.double() / idx.numel() * p.mean(0)).sum(), torch.logsumexp(kept, 1).square().mean()])
        (losses * s["d_losses"].double()).sum().backward()
        return losses.detach(), counts.to(torch.int32), x.grad
    x = _value64(s["x_codes"], s["x_scales"], c["K"]) if c["type"] == "mx4" else s["x"].double()
    if c["op"] == "matmul":
        w = _value64(s["w_codes"], s["w_scales"], c["K"])
        return x @ w if c["grad"] else x @ w.t().contiguous()
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
