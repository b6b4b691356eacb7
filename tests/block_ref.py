"""Plain references of the 8-bit rows and product, the norms around a block and the
group-limited choice of experts, in numpy.  Written from the definitions in
include/weight_only_bit.h; they share no code with the kernels (test_block_ref.py
pins them)."""
import numpy as np

# Half a step of each output type, relative to the value, and half its smallest
# subnormal: what one rounding can be off by.
HALF_STEP = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}
TINY = {"bf16": 2.0 ** -134, "fp16": 2.0 ** -25, "fp32": 2.0 ** -150}

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def int8_rows(v):
    """v [R, K] float32 -> (codes [R, K] int8, scale [R] float32), operation by operation in
    binary32: scale = amax / 127, code = round-half-even(v * (127 / amax)).  (127 / amax
    leaves binary32 for a subnormal amax: there v is taken 2^64 times as large.)"""
    v = np.asarray(v, np.float32)
    with np.errstate(all="ignore"):
        top = np.abs(v).max(-1)
        bad = ~np.isfinite(v).all(-1)
        top = np.where(bad, np.float32(0), top)
        lift = np.where(top < 2.0 ** -100, np.float32(2.0 ** 64), np.float32(1))
        inv = np.where(top > 0, np.float32(127) / (top * lift), np.float32(0)).astype(np.float32)
        scale = np.where(bad, np.float32("nan"), (top / np.float32(127)).astype(np.float32))
        q = np.rint((np.where(bad[:, None], 0, v) * lift[:, None]).astype(np.float32) * inv[:, None])
    return q.astype(np.int8), scale.astype(np.float32)


def silu_mul(x):
    """x [R, 2K] float64 -> silu(gate) * up and how far a binary32 evaluation may be off:
    the exponent's argument is rounded (2^-24 |g|), the exponential off by 2^-22, the sum,
    quotient and product rounded."""
    K = x.shape[1] // 2
    g, u = x[:, :K], x[:, K:]
    with np.errstate(over="ignore"):
        v = g / (1.0 + np.exp(-g)) * u
    return v, np.abs(v) * (2.0 ** -23 * np.abs(g) + 2.0 ** -22 + 5 * 2.0 ** -24) + 2.0 ** -126


def product(xq, xs, wq, ws, bias):
    """(y float64, bound without the output's rounding): the sum is exact; its conversion,
    two products and the bias' addition round (or the last two as one)."""
    s = xq.astype(np.int64) @ wq.astype(np.int64).T
    y = s * xs.astype(np.float64)[:, None] * ws.astype(np.float64)
    bound = 3 * 2.0 ** -24 * np.abs(y)
    if bias is not None:
        y = y + bias.astype(np.float64)
        bound = bound + 2.0 ** -24 * np.abs(y) * 1.001
    return y, bound * 1.001 + 2.0 ** -148


def product_f32(xq, xs, wq, ws):
    """The product without bias, operation by operation in binary32."""
    s = (xq.astype(np.int64) @ wq.astype(np.int64).T).astype(np.float32)
    with np.errstate(all="ignore"):
        return (s * xs[:, None]).astype(np.float32) * ws


# A sum of H squares in binary32 passes through at most this many additions of any one
# term: those of a thread, the lanes' tree and the waves.
CHAIN = 128


def norm(y, r, w, post, gate, alpha, eps):
    """(h, h's bound, n, n's bound) in float64, the bounds without the outputs' own
    rounding.  Each operation in binary32 is off by 2^-24 of its result; a sum of positive
    terms by CHAIN of them, its square root by half of that."""
    u = 2.0 ** -24
    if y is None:
        h, dh = r, np.zeros_like(r)
    else:
        t, dt = y, np.zeros_like(y)
        if post is not None:
            t = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * post
            dt = np.abs(t) * (CHAIN / 2 + 6) * u
        g = alpha * (np.ones_like(y) if gate is None else gate)
        h = r + g * t
        dh = np.abs(g) * dt + 2 * u * np.abs(g * t) + u * np.abs(h)
    if w is None:
        return h, dh, None, None
    ms = (h * h).mean(-1, keepdims=True) + eps
    n = h / np.sqrt(ms) * w
    # the sum moves with h's errors: d(sum h^2) <= 2 |h| |dh|
    ds = (np.abs(h) * dh).mean(-1, keepdims=True) / ms
    dn = np.abs(w) * dh / np.sqrt(ms) + np.abs(n) * ((CHAIN / 2 + 6) * u + ds)
    return h, dh * 1.001 + 2.0 ** -140, n, dn * 1.001 + 2.0 ** -140


def route(logits, topk, bias, sigmoid, groups, topk_groups, group_top, renormalize, scale):
    """(ids [T, topk] int32, weights [T, topk] float64), token by token.  Scores are formed
    in 64 bits and rounded once to binary32, choice values and group values are binary32."""
    T, E = logits.shape
    size = E // groups
    ids = np.full((T, topk), -1, np.int32)
    out = np.zeros((T, topk))
    bias = np.zeros(E, np.float32) if bias is None else bias
    for t in range(T):
        l = logits[t].astype(np.float64)
        l = np.where(np.isnan(l), -np.inf, l)
        with np.errstate(all="ignore"):
            if sigmoid:
                s = 1.0 / (1.0 + np.exp(-l))
            else:
                top = l.max()
                p = np.where(l == top, 1.0, np.exp(l - top)) * (l > -np.inf)
                s = p / max(p.sum(), 1e-300)
            s = s.astype(np.float32)
            c = s + bias
        alive = [e for e in range(E) if l[e] > -np.inf and c[e] > -np.inf]
        value = {}
        for g in range(groups):
            best = sorted((c[e] for e in alive if e // size == g), reverse=True)[:group_top]
            if best:
                value[g] = np.float32(best[0]) + (best[1] if len(best) > 1 else np.float32(0))
        kept = sorted(value, key=lambda g: (-value[g], g))[:topk_groups]
        order = sorted((e for e in alive if e // size in kept), key=lambda e: (-c[e], e))[:topk]
        w = s[order].astype(np.float64)
        if renormalize:
            w = w / w.sum() if w.sum() > 0 else w * 0
        ids[t, :len(order)] = order
        out[t, :len(order)] = w * scale
    return ids, out


def route_bound(w, topk):
    """|weight - w|: the sum of at most topk scores, the quotient and the scale round."""
    return np.abs(w) * (topk + 2) * 2.0 ** -24 + 2.0 ** -148


def mxfp4_values(codes, scale):
    """codes [R, H/2], scale [R, H/32] uint8 -> float64 values and each value's block scale."""
    both = np.stack((codes & 15, codes >> 4), -1).reshape(codes.shape[0], -1)
    s = np.repeat(np.exp2(scale.astype(np.float64) - 127), 32, -1)
    return np.where(both >= 8, -1.0, 1.0) * E2M1[both & 7] * s, s
