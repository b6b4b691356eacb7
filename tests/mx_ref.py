"""Plain 64-bit references of the MXFP4 quantisation and product, the choice of
experts and the mixture-of-experts layer, in numpy.  Written from the
definitions in include/weight_only_bit.h; they share no code with the kernels
(test_mx_ref.py pins them)."""
import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])

# Half a step of each output type, relative to the value, and half its smallest
# subnormal: what one rounding can be off by.
HALF_STEP = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}
TINY = {"bf16": 2.0 ** -134, "fp16": 2.0 ** -25, "fp32": 2.0 ** -150}


def quantize(x):
    """x [R, K] float64 -> (codes [R, K/2] uint8, scale [R, K/32] uint8)."""
    R, K = x.shape
    v = x.reshape(R, K // 32, 32)
    with np.errstate(invalid="ignore"):
        top = np.abs(v).max(-1)
        bad = ~np.isfinite(v).all(-1)
    top = np.where(bad, 0.0, top)
    # frexp: top = m 2^e, m in [1/2, 1), so floor(log2 top) = e - 1
    X = np.where(top > 0, np.frexp(top)[1] - 1 - 2, -127).clip(-127, 127)
    q = np.ldexp(np.where(bad[..., None], 0.0, v), -X[..., None])
    a = np.abs(q)
    d = np.abs(a[..., None] - E2M1)                       # distance to each magnitude
    code = np.zeros(a.shape, np.int64)
    best = np.full(a.shape, np.inf)
    for k in (0, 2, 4, 6, 1, 3, 5, 7):                    # even codes first: they win ties
        closer = d[..., k] < best
        code = np.where(closer, k, code)
        best = np.where(closer, d[..., k], best)
    code = code + 8 * np.signbit(q)
    code = np.where(bad[..., None], 0, code).reshape(R, K).astype(np.uint8)
    scale = np.where(bad, 255, X + 127).astype(np.uint8)
    return code[:, 0::2] | (code[:, 1::2] << 4), scale


def decode(codes, scale):
    """[..., K/2] codes and [..., K/32] scale bytes -> [..., K] float64."""
    c = np.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], -1)
    v = np.where(c >= 8, -1.0, 1.0) * E2M1[c & 7]
    s = np.where(scale == 255, np.nan, np.ldexp(1.0, scale.astype(np.int64) - 127))
    return v * np.repeat(s, 32, -1)


def product(x, xs, w, ws):
    """(y, bound): y [M, N] and, per output, what K fp32 additions (each off by
    at most one step of the running sum, 2^-23, as a truncating adder is) can
    be off by: K 2^-23 sum |x w|."""
    a, b = decode(x, xs), decode(w, ws)
    K = a.shape[1]
    return a @ b.T, K * 2.0 ** -23 * (np.abs(a) @ np.abs(b).T)


def rounded(y, bound, out):
    """Bound on |kernel - y| after one rounding to `out`."""
    return bound * (1 + HALF_STEP[out]) + HALF_STEP[out] * np.abs(y) + TINY[out]


def choose(logits, topk, bias=None, renormalize=True):
    """(ids [T, topk] int32, weights [T, topk] float64, spread [T, topk]): spread
    is max l - l of each chosen place (0 for an empty one)."""
    l = logits.astype(np.float32)
    if bias is not None:
        l = l + bias.astype(np.float32)
    T, E = l.shape
    ids = np.full((T, topk), -1, np.int32)
    w = np.zeros((T, topk))
    spread = np.zeros((T, topk))
    for t in range(T):
        v = [(-np.inf if np.isnan(f) else float(f)) for f in l[t]]
        order = sorted((e for e in range(E) if v[e] > -np.inf), key=lambda e: (-v[e], e))
        if not order:
            continue
        top = v[order[0]]

        def p(e):
            return 1.0 if v[e] == top else float(np.exp(v[e] - top))
        chosen = order[:topk]
        total = sum(p(e) for e in (chosen if renormalize else order))
        for s, e in enumerate(chosen):
            ids[t, s], w[t, s] = e, p(e) / total
            spread[t, s] = 0.0 if v[e] == top else top - v[e]
    return ids, w, spread


def choice_bound(w, spread, E):
    """|weight - w|: the exponential of d = l - max is off by a rounding of d
    (2^-24 d), one of d log2(e) (2^-24 d) and the instruction's own 2^-22; the
    sum of at most E terms by the same and E 2^-24, the quotient by 2^-23.
    Spreads past 126 binary orders come out as zero."""
    d = np.minimum(spread, 128.0).max(-1, keepdims=True)
    return w * (2 * (2.0 ** -23 * d + 2.0 ** -22) + (E + 4) * 2.0 ** -24) + 2.0 ** -125


def layer(x, ids, weights, w1, w1s, w2, w2s):
    """(y, bound) of the mixture-of-experts layer for a given choice.

    The kernel's pre-activations are off by at most H 2^-23 sum |x w1| (fp32
    sums), silu has slope below 1.1, exp and the quotient cost 2^-21, the
    activated row, by itself or weighted, is rounded to bf16 (2^-8), the I
    products and topk slots are summed in fp32, and the weights are off by 2^-18
    (choice_bound for scores within 32 of the maximum and E <= 256)."""
    T, H = x.shape
    I = w2.shape[2] * 2
    y, bound = np.zeros((T, H)), np.zeros((T, H))
    for e in np.unique(ids[ids >= 0]):
        t, s = np.nonzero(ids == e)
        a1, a2 = decode(w1[e], w1s[e]), decode(w2[e], w2s[e])
        pre, off = x[t] @ a1.T, H * 2.0 ** -23 * (np.abs(x[t]) @ np.abs(a1).T)
        g, u = pre[:, :I], pre[:, I:]
        silu = g / (1.0 + np.exp(-g))
        a = silu * u
        da = (1.1 * off[:, :I] * (np.abs(u) + off[:, I:]) + np.abs(silu) * off[:, I:]
              + (2.0 ** -8 + 2.0 ** -21) * np.abs(a) + 2.0 ** -133)
        p = weights[t, s][:, None]
        np.add.at(y, t, p * (a @ a2.T))
        np.add.at(bound, t, p * ((da + (I + ids.shape[1]) * 2.0 ** -23 * np.abs(a) + 2.0 ** -18
                                  * np.abs(a)) @ np.abs(a2).T))
    return y, bound
