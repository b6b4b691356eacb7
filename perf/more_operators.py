"""8-bit rows and their product, the norms around a block, and group-limited expert
routing, as cases that can be timed.

Each case names one pass through one operator.  With ``own`` false ``run``
computes it from elementary torch operations in 32 bits (scores of the routing in
64, because their order decides which experts are taken); with ``own`` true it
makes the calls that a user of weight_only_bit_amd makes.  ``exact`` gives the
same result in 64 bits from the definition.

    quantise  v = x, or silu(gate) * up of a row's halves; one scale a row,
              amax / 127, and codes round(v * 127 / amax); read back as values
    product   y = x_scale[m] * w_scale[n] * sum of int8 products (+ bias[n])
    norm      t = y, or y / rms(y) * post_weight;  h = residual + alpha * gate * t;
              n = h / rms(h) * weight, plain, in int8 rows or in MXFP4 blocks
    route     s = sigmoid or softmax of the scores in binary32, c = s + bias; the
              best groups by the sum of their best one or two c, the best experts
              of those by c, weights from s
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one token's hidden vector before an 8-bit projection: latency only
        dict(name="quantise one token", op="quantise", rows=1, K=5376, act=False, pad=0, dtype="bf16"),
        # gate and up halves of a prefill batch's feed-forward, before the down projection
        dict(name="quantise gated rows", op="quantise", rows=2048, K=21504, act=True, pad=0,
             dtype="bf16"),
        # decode of one token through a qkv projection: the weights' bytes
        dict(name="product one token", op="product", M=1, N=16384, K=5376, out="bf16", bias=False),
        # a small odd batch, K an odd multiple of 64
        dict(name="product 13 tokens", op="product", M=13, N=5760, K=2880, out="fp16", bias=True),
        # a batched decode step through a down projection: between the two bounds
        dict(name="product 100 tokens", op="product", M=100, N=5376, K=21504, out="bf16", bias=False),
        # prefill: matrix-core bound
        dict(name="product prefill", op="product", M=2048, N=16384, K=5376, out="bf16", bias=False),
        # one decoded token between two blocks, into the 4-bit product: latency only
        dict(name="norm one token", op="norm", T=1, H=5376, dtype="bf16", res="bf16", post=True,
             gate="none", out="mxfp4"),
        # a prefill batch with a 32-bit residual stream and a gate per channel, into the 8-bit product
        dict(name="norm prefill", op="norm", T=2048, H=5376, dtype="bf16", res="fp32", post=True,
             gate="channel", out="int8"),
        # a long batch, gated per element (conditioning), 16-bit in and out: memory
        dict(name="norm long batch", op="norm", T=16384, H=5376, dtype="fp16", res="fp16",
             post=False, gate="rows", out="same"),
        # routing of one decoded token: latency only
        dict(name="route one token", op="route", T=1, groups=8, size=32, kept=4, two=True, topk=8,
             dtype="bf16", score="sigmoid", bias=True, renormalize=True, scale=2.5, masked=0),
        # routing of a large prefill batch, some experts masked, padded rows
        dict(name="route many tokens", op="route", T=16384, groups=8, size=32, kept=4, two=True,
             topk=8, dtype="fp32", score="sigmoid", bias=True, renormalize=True, scale=2.5, masked=24),
        # softmax scores, a group's best expert decides, sizes that are no powers of two
        dict(name="route softmax groups", op="route", T=4096, groups=8, size=20, kept=3, two=False,
             topk=6, dtype="bf16", score="softmax", bias=False, renormalize=False, scale=16.0,
             masked=0),
    ]


def _log(rng, lo, hi):
    """A whole number from lo to hi, uniform in its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("quantise", "product", "product", "norm", "norm", "route"))
    if op == "quantise":
        K, act = 16 * _log(rng, 1, 4096), rng.random() < 0.5
        return dict(op=op, rows=_log(rng, 1, min(65536, 2048 * 21504 // K)), K=K, act=act,
                    pad=0 if act else 8 * rng.choice((0, 0, 1, 9, 128)),
                    dtype=rng.choice(("bf16", "fp16", "fp32")))
    if op == "product":
        N, K = 8 * _log(rng, 8, 5376), 16 * _log(rng, 2, 1344)
        while N * K > 43008 * 5376:
            N, K = 8 * _log(rng, 8, 5376), 16 * _log(rng, 2, 1344)
        return dict(op=op, M=_log(rng, 1, min(4096, 2048 * 16384 * 5376 // (N * K))), N=N, K=K,
                    out=rng.choice(("bf16", "bf16", "fp16", "fp32")), bias=rng.random() < 0.5)
    if op == "norm":
        H = 32 * _log(rng, 1, 1024)
        T = _log(rng, 1, min(32768, 16384 * 5376 // H // 2))
        dtype = rng.choice(("bf16", "fp16", "fp32"))
        # 4-bit outputs for decode batches, where the 4-bit product is the better one
        outs = ("same", "int8", "mxfp4") if T * H <= 16 * 5376 else ("same", "int8")
        return dict(op=op, T=T, H=H, dtype=dtype, res=rng.choice((dtype, "fp32")),
                    post=rng.random() < 0.5, gate=rng.choice(("none", "channel", "rows")),
                    out=rng.choice(outs))
    groups, size = rng.choice((1, 2, 4, 8, 16)), _log(rng, 2, 64)
    kept = rng.randint(1, groups)
    return dict(op=op, T=_log(rng, 1, min(32768, 16384 * 256 // (groups * size) // 2)), groups=groups,
                size=size, kept=kept, two=rng.random() < 0.5, topk=rng.randint(1, min(16, kept * size)),
                dtype=rng.choice(("bf16", "fp16", "fp32")), score=rng.choice(("sigmoid", "softmax")),
                bias=rng.random() < 0.7, renormalize=rng.random() < 0.5,
                scale=rng.choice((1.0, 2.5)), masked=rng.choice((0, 0, groups * size // 4)))


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _normal(g, *shape):
    return torch.randn(shape, device="cuda", generator=g)


def _codes(g, *shape):
    """Normal weights or activations in 8 bits, the largest of a row at about 4 sigma."""
    return (_normal(g, *shape) * (127.0 / 4.0)).round_().clamp_(-127, 127).to(torch.int8)


def _scales(g, n, mid):
    return torch.exp(_normal(g, n) * 0.3) * mid


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = dict(case=case, op=case["op"])
    if case["op"] == "quantise":
        R, W = case["rows"], case["K"] * (2 if case["act"] else 1)
        # a hundredth of the columns carries outliers, as activations do
        wide = torch.rand(W + case["pad"], device="cuda", generator=g) < 0.01
        x = torch.where(wide, 10.0, 1.0) * _normal(g, R, W + case["pad"])
        s["x"] = x.to(DT[case["dtype"]])[:, :W]
    elif case["op"] == "product":
        M, N, K = case["M"], case["N"], case["K"]
        s["x"], s["xs"] = _codes(g, M, K), _scales(g, M, 0.03)
        s["w"], s["ws"] = _codes(g, N, K), _scales(g, N, 0.0006)
        s["bias"] = _normal(g, N) if case["bias"] else None
    elif case["op"] == "norm":
        T, H, dt = case["T"], case["H"], DT[case["dtype"]]
        wide = torch.where(torch.rand(H, device="cuda", generator=g) < 0.01, 10.0, 1.0)
        s["y"] = (_normal(g, T, H) * 0.5).to(dt)
        s["r"] = (_normal(g, T, H) * wide).to(DT[case["res"]])
        s["w"] = (1.0 + 0.1 * _normal(g, H)).to(dt)
        s["post"] = (1.0 + 0.1 * _normal(g, H)).to(dt) if case["post"] else None
        shape = dict(none=None, channel=(H,), rows=(T, H))[case["gate"]]
        s["gate"] = None if shape is None else _normal(g, *shape).to(dt)
    else:
        T, E = case["T"], case["groups"] * case["size"]
        v = _normal(g, T, E) * 1.5
        if case["masked"]:  # experts out of service, and one row in 64 a padded one
            v[:, torch.randperm(E, device="cuda", generator=g)[: case["masked"]]] = -math.inf
            v[63::64] = -math.inf
        s["logits"] = v.to(DT[case["dtype"]])
        s["bias"] = _normal(g, E) * 0.1 if case["bias"] else None
    return s


ALPHA, EPS = 0.875, 1e-6  # a residual scale, the norms' epsilon


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def _rows8(v):
    """(bf16 values, scale) of the rows of v (fp32) in 8 bits."""
    top = v.abs().amax(-1, keepdim=True)
    scale = top / 127.0
    q = torch.round(v * torch.where(top > 0, 127.0 / top, 0.0)).clamp_(-127.0, 127.0)
    return (q * scale).to(torch.bfloat16), scale.squeeze(-1)


def _blocks4(x):
    """x's nearest MXFP4 values (per 32: the power of two that puts the largest
    magnitude into [4, 8), elements rounded half to even and held at 6)."""
    v = x.unflatten(-1, (-1, 32))
    top = v.abs().amax(-1, keepdim=True)
    scale = torch.exp2((torch.frexp(top).exponent.float() - 3.0).clamp(-127.0, 127.0))
    q = v.abs() / scale
    step = torch.where(q < 2.0, 0.5, torch.where(q < 4.0, 1.0, 2.0))
    q = (torch.round(q / step) * step).clamp(max=6.0)
    return (torch.copysign(q, v) * scale).flatten(-2).to(torch.bfloat16)


def _route(s, case):
    G, S, K = case["groups"], case["size"], case["topk"]
    l = s["logits"].double()
    out = torch.isnan(l) | (l == -math.inf)
    if case["score"] == "sigmoid":
        p = (1.0 / (1.0 + torch.exp(-l))).float()
    else:
        top = l.amax(-1, keepdim=True)
        p = torch.where(out, 0.0, torch.exp(l - torch.where(top == -math.inf, 0.0, top)))
        p = (p / p.sum(-1, keepdim=True)).float()
    c = p if s["bias"] is None else p + s["bias"]
    c = torch.where(out, -math.inf, c).view(-1, G, S)
    best = torch.sort(c, dim=-1, descending=True).values[..., :2]
    value = best[..., 0]
    if case["two"]:
        value = value + torch.where(best[..., -1] == -math.inf, 0.0, best[..., -1])
    order = torch.sort(value, dim=-1, descending=True, stable=True).indices[:, : case["kept"]]
    keep = torch.zeros(value.shape, dtype=torch.bool, device=l.device).scatter_(1, order, True)
    c = torch.where(keep.unsqueeze(-1), c, -math.inf).flatten(1)
    best, at = torch.sort(c, dim=-1, descending=True, stable=True)
    best, at = best[:, :K], at[:, :K]
    there = best != -math.inf
    w = torch.where(there, p.gather(-1, at), 0.0)
    if case["renormalize"]:
        total = w.sum(-1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    return torch.where(there, at, -1).to(torch.int32), w * case["scale"]


def _own(s, case):
    import weight_only_bit_amd as wob
    if s["op"] == "quantise":
        codes, scale = wob.int8_quantize(s["x"], act=wob.ACT_SILU_MUL if case["act"] else wob.ACT_NONE)
        return wob.int8_dequant(codes, scale, out_dtype=torch.bfloat16), scale
    if s["op"] == "product":
        return wob.int8_gemm(s["x"], s["xs"], s["w"], s["ws"], bias=s["bias"], out_dtype=DT[case["out"]])
    if s["op"] == "norm":
        quant = dict(same=wob.QUANT_NONE, int8=wob.QUANT_INT8, mxfp4=wob.QUANT_MXFP4)[case["out"]]
        got = wob.residual_norm(s["y"], s["r"], s["w"], post_weight=s["post"], gate=s["gate"],
                                alpha=ALPHA, eps=EPS, quant=quant)
        if case["out"] == "same":
            return got
        codes, scale, h = got
        if case["out"] == "int8":
            return wob.int8_dequant(codes, scale, out_dtype=torch.bfloat16), scale, h
        return wob.mxfp4_dequant(codes, scale), h
    return wob.moe_route(s["logits"], case["topk"], bias=s["bias"],
                         score=wob.SCORE_SIGMOID if case["score"] == "sigmoid" else wob.SCORE_SOFTMAX,
                         groups=case["groups"], topk_groups=case["kept"],
                         group_top=2 if case["two"] else 1, renormalize=case["renormalize"],
                         scale=case["scale"])


def run(s):
    case = s["case"]
    if own:
        return _own(s, case)
    if s["op"] == "quantise":
        v = s["x"].float()
        if case["act"]:
            gate, up = v[:, : case["K"]], v[:, case["K"]:]
            v = gate / (1.0 + torch.exp(-gate)) * up
        return _rows8(v)
    if s["op"] == "product":
        y = s["x"].float() @ s["w"].float().t() * s["xs"].unsqueeze(1) * s["ws"]
        return (y if s["bias"] is None else y + s["bias"]).to(DT[case["out"]])
    if s["op"] == "norm":
        t = s["y"].float()
        if case["post"]:
            t = t * torch.rsqrt((t * t).mean(-1, keepdim=True) + EPS) * s["post"].float()
        h = s["r"].float() + t * (ALPHA if s["gate"] is None else ALPHA * s["gate"].float())
        n = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * s["w"].float()
        h = h.to(DT[case["res"]])
        if case["out"] == "same":
            return n.to(DT[case["dtype"]]), h
        return (*_rows8(n), h) if case["out"] == "int8" else (_blocks4(n), h)
    return _route(s, case)


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    if case["op"] == "quantise":  # x in, the bf16 values and a scale a row out; a maximum and a rounding each
        n = case["rows"] * case["K"]
        return dict(bytes=n * (SIZE[case["dtype"]] * (2 if case["act"] else 1) + 2) + 4 * case["rows"],
                    flops=(8 if case["act"] else 2) * n)
    if case["op"] == "product":
        M, N, K = case["M"], case["N"], case["K"]
        return dict(bytes=(M + N) * (K + 4) + M * N * SIZE[case["out"]] + (4 * N if case["bias"] else 0),
                    flops=2 * M * N * K)
    if case["op"] == "norm":  # y, the residual in and out, a gate per element, the normed rows
        n, dt = case["T"] * case["H"], SIZE[case["dtype"]]
        per = dt + 2 * SIZE[case["res"]] + (dt if case["gate"] == "rows" else 0) + (dt if case["out"] == "same" else 2)
        return dict(bytes=n * per, flops=n * (10 if case["post"] else 6))
    n = case["T"] * case["groups"] * case["size"]
    return dict(bytes=n * SIZE[case["dtype"]] + 8 * case["T"] * case["topk"], flops=6 * n)


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------

def _rows8_64(v):
    scale = v.abs().max(dim=-1, keepdim=True).values / 127.0
    code = torch.where(scale > 0, v / scale, 0.0)
    low = torch.floor(code)
    up = (code - low > 0.5) | ((code - low == 0.5) & (torch.remainder(low, 2.0) == 1.0))
    return (low + up.double()) * scale, scale[:, 0]


def _blocks4_64(v):
    """The nearest E2M1 magnitude by the borders between neighbours; a value on a
    border goes to the neighbour with the even code."""
    table = torch.tensor((0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0), dtype=torch.float64, device=v.device)
    shape, v = v.shape, v.reshape(-1, 32)
    top = v.abs().max(dim=-1, keepdim=True).values
    e = torch.floor(torch.log2(top))
    e = e + (torch.exp2(e + 1) <= top).double() - (torch.exp2(e) > top).double()
    e = torch.where(top > 0, e - 2, -127.0).clamp(-127, 127)
    q = torch.ldexp(v.abs(), -e).unsqueeze(-1)
    border, odd = (table[1:] + table[:-1]) / 2, torch.arange(7, device=v.device) % 2 == 1
    code = ((q > border) | ((q == border) & odd)).sum(-1)
    return (torch.ldexp(table[code], e) * torch.where(v < 0, -1.0, 1.0)).reshape(shape)


def _route64(s, case):
    """One place after the other, the first of the largest left; scores and choice
    values are binary32 numbers by definition."""
    G, S = case["groups"], case["size"]
    l = s["logits"].double()
    gone = ~(l > -math.inf)
    if case["score"] == "sigmoid":
        p = 0.5 * (1.0 + torch.tanh(0.5 * l))
        small = l < -1.0  # where the sum above cancels
        p = torch.where(small, torch.exp(l) / (1.0 + torch.exp(l)), p)
    else:
        p = torch.exp(l - torch.logsumexp(l, -1, keepdim=True))
    p = p.float()
    c = (p if s["bias"] is None else p + s["bias"]).masked_fill(gone, -math.inf)
    first, rest = [], c.view(-1, G, S).clone()
    for _ in range(2 if case["two"] else 1):
        if S > len(first):
            top, at = rest.max(-1, keepdim=True)
            first.append(top.squeeze(-1))
            rest.scatter_(-1, at, -math.inf)
    value = first[0] + (first[1].masked_fill(first[1] == -math.inf, 0.0) if len(first) > 1 else 0.0)
    closed = torch.ones_like(value, dtype=torch.bool)
    left = value.clone()
    for _ in range(case["kept"]):
        at = (left == left.amax(-1, keepdim=True)).int().argmax(-1, keepdim=True)
        closed.scatter_(-1, at, False)
        left.scatter_(-1, at, -math.inf)
    left = c.masked_fill(closed.repeat_interleave(S, -1), -math.inf)
    ids, weights = [], []
    for _ in range(case["topk"]):
        best = left.amax(-1, keepdim=True)
        at = (left == best).int().argmax(-1, keepdim=True)
        none = best == -math.inf
        ids.append(at.masked_fill(none, -1))
        weights.append(p.double().gather(-1, at).masked_fill(none, 0.0))
        left.scatter_(-1, at, -math.inf)
    ids, weights = torch.cat(ids, -1), torch.cat(weights, -1)
    if case["renormalize"]:
        total = weights.sum(-1, keepdim=True)
        weights = torch.where(total > 0, weights / total, 0.0)
    return ids.to(torch.int32), weights * case["scale"]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantise":
        v = s["x"].double()
        if case["act"]:
            v = v[:, : case["K"]] * torch.special.expit(v[:, : case["K"]]) * v[:, case["K"]:]
        return _rows8_64(v)
    if case["op"] == "product":
        y = torch.matmul(s["x"].double(), s["w"].double().t())
        y *= s["xs"].double()[:, None]
        y *= s["ws"].double()[None, :]
        return y if s["bias"] is None else y + s["bias"].double()
    if case["op"] == "norm":
        t = s["y"].double()
        if case["post"]:
            t = t / torch.sqrt(t.pow(2).sum(-1, keepdim=True) / case["H"] + EPS) * s["post"].double()
        if s["gate"] is not None:
            t = t * s["gate"].double()
        h = s["r"].double() + ALPHA * t
        n = h / torch.sqrt(h.pow(2).sum(-1, keepdim=True) / case["H"] + EPS) * s["w"].double()
        if case["out"] == "same":
            return n, h
        return (*_rows8_64(n), h) if case["out"] == "int8" else (_blocks4_64(n), h)
    return _route64(s, case)
