"""The MXFP4 quantisation, the MXFP4 x MXFP4 product, the expert choice and the
mixture-of-experts layer for a few tokens, as cases that can be timed.

Each case names one pass through one operator.  With ``own`` false ``run``
computes it from elementary torch operations in 32 bits; with ``own`` true it
makes the calls that a user of weight_only_bit_amd makes.  ``exact`` gives the
same result in 64 bits from the definition.

Formats: E2M1 codes, two per byte (the even element in the low nibble), one
E8M0 byte b per 32 elements of a row (scale 2^(b - 127)).
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}

# The magnitudes of E2M1 codes 0..7 (code + 8 is the negative).
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one token's hidden vector before a 4-bit projection: latency only
        dict(name="quantise one token", op="quantise", rows=1, K=5376, pad=0, dtype="bf16"),
        # a prefill batch's activations, a column slice of a wider buffer (fused projection)
        dict(name="quantise prefill rows", op="quantise", rows=2048, K=5376, pad=512, dtype="fp16"),
        # a checkpoint's 32-bit projection matrix turned into weights
        dict(name="quantise a weight", op="quantise", rows=16384, K=5376, pad=0, dtype="fp32"),
        # decode of one token through a qkv projection: the weights' bytes
        dict(name="product one token", op="product", M=1, N=16384, K=5376, out="bf16"),
        # a small odd batch, K an odd multiple of 64
        dict(name="product 13 tokens", op="product", M=13, N=5760, K=2880, out="fp16"),
        # a batched decode step through a down projection: between the two bounds
        dict(name="product 100 tokens", op="product", M=100, N=5376, K=21504, out="bf16"),
        # prefill: matrix-core bound
        dict(name="product prefill", op="product", M=2048, N=16384, K=5376, out="bf16"),
        # expert choice of one decoded token: latency only
        dict(name="choice one token", op="choice", T=1, E=32, topk=4, dtype="bf16", bias=True,
             renormalize=True, masked=0),
        # expert choice of a large prefill batch over many experts, some of them masked
        dict(name="choice many tokens", op="choice", T=16384, E=256, topk=8, dtype="fp32",
             bias=False, renormalize=False, masked=24),
        # a mixture-of-experts layer for one decoded token
        dict(name="layer one token", op="layer", T=1, E=32, topk=4, H=2880, I=2880, dtype="bf16",
             bias=True, renormalize=True),
        # the same for a small batch
        dict(name="layer 4 tokens", op="layer", T=4, E=32, topk=4, H=2880, I=2880, dtype="bf16",
             bias=True, renormalize=True),
        # the same for a batch that reaches every expert
        dict(name="layer 32 tokens", op="layer", T=32, E=32, topk=4, H=2880, I=2880, dtype="fp32",
             bias=False, renormalize=True),
    ]


def _log(rng, lo, hi):
    """A whole number from lo to hi, uniform in its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("quantise", "product", "product", "choice", "layer"))
    if op == "quantise":
        K = 32 * _log(rng, 1, 672)
        return dict(op=op, rows=_log(rng, 1, min(65536, 16384 * 5376 // K)), K=K,
                    pad=8 * rng.choice((0, 0, 1, 9, 128)),
                    dtype=rng.choice(("bf16", "fp16", "fp32")))
    if op == "product":
        N, K = 8 * _log(rng, 8, 5376), 32 * _log(rng, 2, 672)
        while N * K > 43008 * 5376:
            N, K = 8 * _log(rng, 8, 5376), 32 * _log(rng, 2, 672)
        return dict(op=op, M=_log(rng, 1, min(4096, 2048 * 16384 * 5376 // (N * K))), N=N, K=K,
                    out=rng.choice(("bf16", "bf16", "fp16", "fp32")))
    if op == "choice":
        E = _log(rng, 4, 512)
        return dict(op=op, T=_log(rng, 1, min(65536, 16384 * 256 // E // 2)), E=E,
                    topk=rng.randint(1, min(16, E)), dtype=rng.choice(("bf16", "fp16", "fp32")),
                    bias=rng.random() < 0.5, renormalize=rng.random() < 0.5,
                    masked=rng.choice((0, 0, E // 4)))
    E = _log(rng, 4, 64)
    H, I = 64 * _log(rng, 4, 48), 64 * _log(rng, 4, 48)
    while E * H * I > 32 * 2880 * 2880:
        H, I = 64 * _log(rng, 4, 48), 64 * _log(rng, 4, 48)
    return dict(op=op, T=_log(rng, 1, 32), E=E, topk=rng.randint(1, min(8, E)), H=H, I=I,
                dtype=rng.choice(("bf16", "fp32")), bias=rng.random() < 0.5,
                renormalize=rng.random() < 0.5)


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _codes(g, *shape):
    return torch.randint(0, 256, shape, dtype=torch.uint8, device="cuda", generator=g)


def _scales(g, lo, hi, *shape):
    return torch.randint(lo, hi + 1, shape, dtype=torch.uint8, device="cuda", generator=g)


def _logits(g, T, E, case, masked):
    """Router scores; `masked` experts hold -inf, and with a mask one row in 64
    has no expert left (a padded row of the batch)."""
    v = torch.randn((T, E), device="cuda", generator=g) * 1.5
    if masked:
        v[:, torch.randperm(E, device="cuda", generator=g)[:masked]] = -math.inf
        v[63::64] = -math.inf
    bias = torch.randn(E, device="cuda", generator=g) * 0.5 if case["bias"] else None
    return v.to(DT[case["dtype"]]), bias


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = dict(case=case, op=case["op"])
    # the values of a byte's two codes, for the plain form
    half = torch.tensor(E2M1 + tuple(-v for v in E2M1), device="cuda")
    s["pairs"] = torch.stack((half.repeat(16), half.repeat_interleave(16)), 1)
    if case["op"] == "quantise":
        R, K = case["rows"], case["K"]
        x = torch.randn((R, K + case["pad"]), device="cuda", generator=g)
        # a hundredth of the columns carries outliers, as activations do
        wide = torch.rand(K + case["pad"], device="cuda", generator=g) < 0.01
        x = torch.where(wide, x * 50.0, x)
        s["x"] = x.to(DT[case["dtype"]])[:, :K]
    elif case["op"] == "product":
        M, N, K = case["M"], case["N"], case["K"]
        s["x"], s["xs"] = _codes(g, M, K // 2), _scales(g, 124, 128, M, K // 32)
        s["w"], s["ws"] = _codes(g, N, K // 2), _scales(g, 117, 121, N, K // 32)
    elif case["op"] == "choice":
        s["logits"], s["bias"] = _logits(g, case["T"], case["E"], case, case["masked"])
    else:
        T, E, H, I = case["T"], case["E"], case["H"], case["I"]
        s["x"] = torch.randn((T, H), device="cuda", generator=g).to(torch.bfloat16)
        s["logits"], s["bias"] = _logits(g, T, E, case, 0)
        s["w1"], s["w1s"] = _codes(g, E, 2 * I, H // 2), _scales(g, 117, 121, E, 2 * I, H // 32)
        s["w2"], s["w2s"] = _codes(g, E, H, I // 2), _scales(g, 117, 121, E, H, I // 32)
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def _values(pairs, codes, scales):
    """The fp32 values of packed codes [..., K/2] under E8M0 scales [..., K/32]."""
    v = pairs[codes.int()].flatten(-2)
    return (v.unflatten(-1, (-1, 32)) * torch.exp2(scales.float() - 127.0).unsqueeze(-1)).flatten(-2)


def _quantised(x):
    """x's nearest MXFP4 values (per 32: the power of two that puts the largest
    magnitude into [4, 8), elements rounded half to even and held at 6)."""
    v = x.float().unflatten(-1, (-1, 32))
    top = v.abs().amax(-1, keepdim=True)
    e = (torch.frexp(top).exponent.float() - 3.0).clamp(-127.0, 127.0)
    scale = torch.exp2(e)
    q = v.abs() / scale
    step = torch.where(q < 2.0, 0.5, torch.where(q < 4.0, 1.0, 2.0))
    q = (torch.round(q / step) * step).clamp(max=6.0)
    return (torch.copysign(q, v) * scale).flatten(-2).to(torch.bfloat16)


def _chosen(logits, bias, topk, renormalize):
    """The topk largest scores of each row (ties to the lowest index) and their
    softmax weights; places without a score hold id -1 and weight 0."""
    v = logits.float() if bias is None else logits.float() + bias
    v = torch.where(torch.isnan(v), -math.inf, v)
    best, at = torch.sort(v, dim=-1, descending=True, stable=True)
    top = best[:, :1]
    p = torch.where(v == -math.inf, 0.0, torch.exp(v - top))
    best, at = best[:, :topk], at[:, :topk]
    there = best != -math.inf
    w = torch.where(there, torch.exp(best - top), 0.0)
    total = (w if renormalize else p).sum(-1, keepdim=True)
    return (torch.where(there, at, -1).to(torch.int32),
            torch.where(there, w / total, 0.0))


def _layer(s, case):
    E, H, I, T = case["E"], case["H"], case["I"], case["T"]
    ids, weights = _chosen(s["logits"], s["bias"], case["topk"], case["renormalize"])
    share = torch.zeros((T, E), device="cuda").scatter_(1, ids.long(), weights)
    w1 = _values(s["pairs"], s["w1"], s["w1s"]).view(E * 2 * I, H)
    h = (s["x"].float() @ w1.t()).view(T, E, 2, I)
    h = torch.sigmoid(h[:, :, 0]) * h[:, :, 0] * h[:, :, 1] * share.unsqueeze(-1)
    w2 = _values(s["pairs"], s["w2"], s["w2s"]).permute(1, 0, 2).reshape(H, E * I)
    return (h.view(T, E * I) @ w2.t()).to(torch.bfloat16)


def run(s):
    case = s["case"]
    if own:
        import weight_only_bit_amd as wob
        if s["op"] == "quantise":
            return wob.mxfp4_dequant(*wob.mxfp4_quantize(s["x"]))
        if s["op"] == "product":
            return wob.mxfp4_gemm(s["x"], s["xs"], s["w"], s["ws"], out_dtype=DT[case["out"]])
        if s["op"] == "choice":
            return wob.moe_topk(s["logits"], case["topk"], bias=s["bias"],
                                renormalize=case["renormalize"])
        return wob.mxfp4_moe_layer(s["x"], s["logits"], case["topk"], s["w1"], s["w1s"], s["w2"],
                                   s["w2s"], bias=s["bias"], renormalize=case["renormalize"])
    if s["op"] == "quantise":
        return _quantised(s["x"])
    if s["op"] == "product":
        x, w = _values(s["pairs"], s["x"], s["xs"]), _values(s["pairs"], s["w"], s["ws"])
        return (x @ w.t()).to(DT[case["out"]])
    if s["op"] == "choice":
        return _chosen(s["logits"], s["bias"], case["topk"], case["renormalize"])
    return _layer(s, case)


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    size = {"bf16": 2, "fp16": 2, "fp32": 4}
    if case["op"] == "quantise":  # x in, the bf16 values out; a maximum and a rounding each
        n = case["rows"] * case["K"]
        return dict(bytes=n * (size[case["dtype"]] + 2), flops=2 * n)
    if case["op"] == "product":  # codes and scales in, the product out
        M, N, K = case["M"], case["N"], case["K"]
        return dict(bytes=(M + N) * (K // 2 + K // 32) + M * N * size[case["out"]],
                    flops=2 * M * N * K)
    T, E, topk = case["T"], case["E"], case["topk"]
    if case["op"] == "choice":
        return dict(bytes=T * E * size[case["dtype"]] + (4 * E if case["bias"] else 0) + 8 * T * topk,
                    flops=3 * T * E)
    # the weights of the experts that T tokens reach on average
    H, I = case["H"], case["I"]
    reached = E * (1.0 - (1.0 - topk / E) ** T)
    return dict(bytes=int(reached * 3 * I * H * (0.5 + 1 / 32)) + 4 * T * H + T * E * size[case["dtype"]],
                flops=2 * T * topk * 3 * I * H)


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------

def _decode64(codes, scales):
    """Values from the bit fields: (-1)^s 2^(e-1) (1 + m/2), or m/2 where e = 0."""
    both = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    e, m = ((both >> 1) & 3).double(), (both & 1).double()
    v = torch.where(e == 0, 0.5 * m, torch.ldexp(1.0 + 0.5 * m, e - 1.0))
    v = torch.where(both >= 8, -v, v)
    return v * torch.ldexp(torch.ones((), dtype=torch.float64, device=v.device),
                           scales.double() - 127.0).repeat_interleave(32, -1)


def _choice64(v, topk, renormalize):
    """The choice one place after the other: the first of the largest left."""
    v = torch.nan_to_num(v, nan=-math.inf, posinf=math.inf, neginf=-math.inf)
    top = v.amax(-1, keepdim=True)
    p = torch.exp(v - torch.where(top == -math.inf, 0.0, top))
    left, ids, weights = v.clone(), [], []
    for _ in range(topk):
        best = left.amax(-1, keepdim=True)
        at = (left == best).int().argmax(-1, keepdim=True)
        none = best == -math.inf
        ids.append(torch.where(none, -1, at))
        weights.append(torch.where(none, 0.0, p.gather(-1, at)))
        left.scatter_(-1, at, -math.inf)
    ids, weights = torch.cat(ids, -1), torch.cat(weights, -1)
    total = (weights if renormalize else p).sum(-1, keepdim=True)
    return ids, torch.where(total > 0, weights / total, 0.0)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantise":
        # the nearest E2M1 magnitude by the borders between neighbours; a value
        # on a border goes to the neighbour with the even code
        v = s["x"].double().unflatten(-1, (-1, 32))
        top = v.abs().amax(-1, keepdim=True)
        e = torch.floor(torch.log2(top))
        e = e + (torch.exp2(e + 1) <= top).double() - (torch.exp2(e) > top).double()
        e = torch.where(top > 0, e - 2, -127.0).clamp(-127, 127)
        q = torch.ldexp(v.abs(), -e)
        code = torch.zeros_like(q)
        for k in range(7):
            border = (E2M1[k] + E2M1[k + 1]) / 2
            code += ((q > border) | ((q == border) & (k % 2 == 1))).double()
        table = torch.tensor(E2M1, dtype=torch.float64, device=q.device)
        return (torch.ldexp(table[code.long()], e) * torch.where(v < 0, -1.0, 1.0)).flatten(-2)
    if case["op"] == "product":
        return _decode64(s["x"], s["xs"]) @ _decode64(s["w"], s["ws"]).t()
    v = s["logits"].float() if s["bias"] is None else s["logits"].float() + s["bias"]
    ids, weights = _choice64(v.double(), case["topk"], case["renormalize"])
    if case["op"] == "choice":
        return ids.to(torch.int32), weights
    y = torch.zeros((case["T"], case["H"]), dtype=torch.float64, device="cuda")
    for e in range(case["E"]):
        token, slot = torch.nonzero(ids == e, as_tuple=True)
        if token.numel():
            gu = s["x"][token].double() @ _decode64(s["w1"][e], s["w1s"][e]).t()
            gate, up = gu[:, : case["I"]], gu[:, case["I"]:]
            a = gate / (1.0 + torch.exp(-gate)) * up
            y.index_add_(0, token, (a @ _decode64(s["w2"][e], s["w2s"][e]).t())
                         * weights[token, slot].unsqueeze(-1))
    return y
