"""Pins of the plain references in mx_ref.py (CPU)."""
import numpy as np
import pytest

from tests import mx_ref as R


def test_decode_agrees_with_the_oracle(oracle):
    codes = np.arange(256, dtype=np.uint8).reshape(1, 256)
    scale = np.full((1, 16), 127, np.uint8)
    want = np.stack((oracle.e2m1_decode(codes[0] & 15), oracle.e2m1_decode(codes[0] >> 4)), -1)
    assert np.array_equal(R.decode(codes, scale)[0], want.reshape(-1).astype(np.float64))
    b = np.arange(255, dtype=np.uint8)
    one = np.full((255, 16), 0x22, np.uint8)  # every element 1.0
    assert np.array_equal(R.decode(one, b[:, None])[:, 0], oracle.e8m0_decode(b).astype(np.float64))


def test_quantize_hand_block():
    """amax 6 -> X = 0; ties to the even code; 5 goes to 4, 7/8 of a step holds at 6."""
    v = np.zeros((1, 32))
    v[0, :16] = [6, -6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, 0.26, -5.01, 4.99, 0.1, -0.1, 1]
    codes, scale = R.quantize(v)
    got = R.decode(codes, scale)[0, :16]
    assert scale[0, 0] == 127
    assert got.tolist() == [6, -6, 0, 1, 1, 2, 2, 4, 4, 0, 0.5, -6, 4, 0, 0, 1]
    nib = np.stack((codes & 15, codes >> 4), -1).reshape(-1)
    assert nib[9] == 8 and nib[14] == 8  # the sign of a value that rounds to zero is kept
    v[0, 0] = 7.9  # still X = 0: held at 6
    assert R.decode(*R.quantize(v))[0, 0] == 6.0
    v[0, 0] = 8.0
    assert R.quantize(v)[1][0, 0] == 128


@pytest.mark.parametrize("mag,byte", [(0.0, 0), (2.0 ** -149, 0), (2.0 ** -126, 0), (2.0 ** -125, 0),
                                      (2.0 ** -124, 1), (1.0, 125), (2.0 ** 127, 252),
                                      (np.inf, 255), (np.nan, 255)])
def test_quantize_scale_byte(mag, byte):
    v = np.zeros((1, 64))
    v[0, 40] = mag
    codes, scale = R.quantize(v)
    assert scale.tolist() == [[0, byte]]
    if byte == 255:
        assert not codes.any()


def test_quantize_is_nearest():
    """No E2M1 value of the block's scale is nearer than the chosen one."""
    rng = np.random.default_rng(0)
    v = rng.standard_normal((50, 64)) * np.exp2(rng.integers(-20, 20, (50, 1)))
    codes, scale = R.quantize(v)
    got = R.decode(codes, scale)
    grid = np.concatenate((R.E2M1, -R.E2M1))
    s = np.repeat(np.exp2(scale.astype(float) - 127), 32, -1)
    best = np.abs(v[..., None] - grid * s[..., None]).min(-1)
    assert np.array_equal(np.abs(v - got), best)
    amax = np.abs(v.reshape(50, 2, 32)).max(-1) / np.exp2(scale.astype(float) - 127)
    assert (amax >= 4).all() and (amax < 8).all()


def test_product_bound_catches_a_swapped_nibble():
    rng = np.random.default_rng(1)
    x, w = rng.integers(0, 256, (4, 64), np.uint8), rng.integers(0, 256, (8, 64), np.uint8)
    xs, ws = np.full((4, 4), 126, np.uint8), np.full((8, 4), 120, np.uint8)
    y, bound = R.product(x, xs, w, ws)
    swapped, _ = R.product((x >> 4) | (x << 4), xs, w, ws)
    assert (np.abs(swapped - y) > R.rounded(y, bound, "bf16")).mean() > 0.5


def test_choose_hand_rows():
    inf, nan = np.inf, np.nan
    l = np.array([[1, 3, 3, 2], [-inf, -inf, -inf, -inf], [nan, 0, -inf, -inf], [inf, 5, inf, 1],
                  [0.0, -0.0, -1, -1]], np.float32)
    ids, w, _ = R.choose(l, 3)
    assert ids.tolist() == [[1, 2, 3], [-1, -1, -1], [1, -1, -1], [0, 2, 1], [0, 1, 2]]
    e = np.exp(-1.0)
    assert np.allclose(w[0], np.array([1, 1, e]) / (2 + e))
    assert w[1].tolist() == [0, 0, 0] and w[2].tolist() == [1, 0, 0]
    assert w[3].tolist() == [0.5, 0.5, 0]
    ids, w, _ = R.choose(l, 2, renormalize=False)
    assert np.allclose(w[0], np.array([1, 1]) / (2 + e + np.exp(-2.0)))
    ids, _, _ = R.choose(l[:1], 1, bias=np.array([9, 0, 0, 0], np.float32))
    assert ids.tolist() == [[0]]


def test_layer_of_one_expert_is_a_gated_product():
    rng = np.random.default_rng(2)
    H, I, T = 64, 64, 3
    w1, w2 = rng.integers(0, 256, (1, 2 * I, H // 2), np.uint8), rng.integers(0, 256, (1, H, I // 2), np.uint8)
    w1s, w2s = np.full((1, 2 * I, 2), 120, np.uint8), np.full((1, H, 2), 120, np.uint8)
    x = rng.standard_normal((T, H))
    y, bound = R.layer(x, np.zeros((T, 1), np.int32), np.ones((T, 1)), w1, w1s, w2, w2s)
    pre = x @ R.decode(w1[0], w1s[0]).T
    g, u = pre[:, :I], pre[:, I:]
    want = (g / (1 + np.exp(-g)) * u) @ R.decode(w2[0], w2s[0]).T
    assert np.allclose(y, want, rtol=1e-12, atol=0)
    assert (bound < 0.05 * np.abs(want).max()).all()
