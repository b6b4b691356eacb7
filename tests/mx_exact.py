"""Operands whose results hold in binary32 whatever the order of the sums, and those
results: a block, a part of K, a place or a scale that is left out or misplaced shows as
a difference, where the bound on K roundings of a random sum hides it (at K = 475168 it
is twelve times the result).  test_mx_exact.py pins both."""
import numpy as np

from tests import mx_ref as R


def _pack(codes):
    return (codes[..., 0::2] | codes[..., 1::2] << 4).astype(np.uint8)


def _codes(rng, magnitudes, shape, signed=True):
    """Codes of whole magnitudes, none of them zero."""
    of = {1: 2, 2: 4, 3: 5, 4: 6, 6: 7}
    c = np.array([of[m] for m in magnitudes], np.uint8)[rng.integers(0, len(magnitudes), shape, np.uint8)]
    return c | rng.integers(0, 2, shape, np.uint8) << 3 if signed else c


def product_operands(M, N, K, seed):
    """Whole numbers under scales of 1 and 2, no code a zero."""
    rng = np.random.default_rng(seed)
    return (_pack(_codes(rng, (1, 2, 3, 4, 6), (M, K))), rng.integers(127, 129, (M, K // 32), np.uint8),
            _pack(_codes(rng, (1, 2), (N, K))), rng.integers(127, 129, (N, K // 32), np.uint8))


def product(x, xs, w, ws):
    """y in float64; every sum of its terms in any order is a whole number below 2^24."""
    a, b = R.decode(x, xs), R.decode(w, ws)
    assert (np.abs(a) @ np.abs(b).T).max() < 2.0 ** 24
    return a @ b.T


def bf16(v):
    """v (float64 that binary32 holds) rounded to bfloat16, ties to even, as float64."""
    f = v.astype(np.float32)
    assert np.array_equal(f.astype(np.float64), v)
    u = f.view(np.uint32).astype(np.uint64)
    u = (u + 0x7FFF + (u >> 16 & 1)) & 0xFFFF0000
    return u.astype(np.uint32).view(np.float32).astype(np.float64)


def _sparse(rng, shape, first_last, share, magnitudes, signed):
    """Codes [..., K] that are zero but for one of a block of 32: in a `share` of the blocks,
    and in the first and the last."""
    *lead, K = shape
    KB = K // 32
    on = rng.random((*lead, KB)) < share
    if first_last:
        on[..., 0] = on[..., -1] = True
    c = np.zeros((*lead, KB, 32), np.uint8)
    at = rng.integers(0, 32, (*lead, KB, 1))
    np.put_along_axis(c, at, np.where(on, _codes(rng, magnitudes, (*lead, KB), signed), 0)[..., None], -1)
    return c.reshape(shape)


def layer_operands(T, E, topk, H, I, seed):
    """(x, logits, weights) float64, float32 and codes.  x is positive and gate codes are too,
    so silu(gate) is gate itself; a token's experts, a power of two in number, have equal
    scores, so their weights are exact."""
    rng = np.random.default_rng(seed)
    n = max(1, min(32, 128 // (H // 32)))               # of a block of x
    x = np.zeros((T, H // 32, 32))
    x[..., :n] = rng.integers(1, 3, (T, H // 32, n))
    x = rng.permuted(x, axis=-1).reshape(T, H)
    places = 1 << topk.bit_length() - 1
    logits = np.full((T, E), -np.inf if places < topk else -1.0, np.float32)
    for t in range(T):
        logits[t, rng.permutation(E)[:places]] = 1.0
    w1 = np.concatenate((_codes(rng, (1, 2, 3), (E, I, H), False), _codes(rng, (1, 2, 3), (E, I, H))), 1)
    w2 = _sparse(rng, (E, H, I), True, min(1.0, max(2, 32 // places) / (I // 32)), (1, 2), True)
    return x, logits, (_pack(w1), rng.integers(127, 129, (E, 2 * I, H // 32), np.uint8),
                       _pack(w2), rng.integers(127, 129, (E, H, I // 32), np.uint8))


def layer(x, logits, topk, w1, w1s, w2, w2s, ids=None):
    """y [T, H] in float64, rounded to bf16 as the layer rounds: the activated rows, then y."""
    if ids is None:
        ids, p, _ = R.choose(logits, topk)
        assert set(np.unique(p)) <= {0.0, p.max()}
    share = 1.0 / (1 << topk.bit_length() - 1)
    T, I = x.shape[0], w2.shape[2] * 2
    y, most, unit = np.zeros((T, w2.shape[1])), np.zeros((T, w2.shape[1])), np.inf
    for e in np.unique(ids[ids >= 0]):
        t = np.nonzero(ids == e)[0]
        pre = x[t] @ R.decode(w1[e], w1s[e]).T
        g, u = pre[:, :I], pre[:, I:]
        # exp(-g) is below half a step of 1, so silu(g) = g; g u is a whole number below 2^24
        assert g.min() > 18 and np.abs(g * u).max() < 2.0 ** 24 and np.abs(pre).max() < 2.0 ** 24
        a = bf16(share * g * u)
        b = R.decode(w2[e], w2s[e])
        y[t] += a @ b.T
        most[t] += np.abs(a) @ np.abs(b).T
        m, x2 = np.frexp(np.abs(a[a != 0]))
        low = (m * 256).astype(np.int64)                # the eight bits of a bf16
        unit = min(unit, np.ldexp((low & -low).astype(np.float64), x2 - 8).min(initial=np.inf))
    assert most.max() < 2.0 ** 24 * unit                # every sum in units of the smallest step
    return bf16(y)
