"""Pins of the exact operands of mx_exact.py (CPU): their sums are exact, and what a kernel
could leave out shows."""
import numpy as np
import pytest

from tests import mx_exact as X

# every length of the GPU tests, few rows and columns
LENGTHS = [32, 96, 352, 512, 1056, 4960, 8160, 8224, 9152, 21504, 53600, 65536, 131072, 453664, 475168]
LAYERS = [(1, 8, 4, 2880, 2880), (4, 8, 4, 576, 448), (1, 2, 2, 32832, 64), (1, 2, 2, 64, 32768), (4, 16, 16, 64, 64),
          (3, 5, 3, 192, 320), (8, 70, 64, 64, 64), (1, 4, 1, 1088, 64), (8, 2, 2, 64, 9024)]


@pytest.mark.parametrize("K", LENGTHS)
def test_product_shows_what_is_left_out(K):
    x, xs, w, ws = X.product_operands(3, 40, K, K)
    y = X.product(x, xs, w, ws)

    def differs(*ops):
        return (X.product(*ops) != y).mean()
    assert (y != 0).mean() > 0.9                        # zeros in place of y
    for left in {32, K // 16 // 32 * 32, K // 2 // 32 * 32} - {0, K}:   # a block, a part, half of K
        assert differs(x[:, :(K - left) // 2], xs[:, :(K - left) // 32], w[:, :(K - left) // 2],
                       ws[:, :(K - left) // 32]) > 0.9, left
        assert differs(x[:, left // 2:], xs[:, left // 32:], w[:, left // 2:], ws[:, left // 32:]) > 0.9
    if K > 512:                                         # scales of the neighbouring block or span
        assert differs(x, np.roll(xs, 1, 1), w, ws) > 0.9
        assert differs(x, xs, w, np.roll(ws, 16, 1)) > 0.9
        one = ws.copy()
        one[:, -1] ^= 127 ^ 128                         # of the last block alone
        assert differs(x, xs, w, one) > 0.9


@pytest.mark.parametrize("T,E,topk,H,I", LAYERS)
def test_layer_shows_what_is_left_out(T, E, topk, H, I):
    x, logits, w = X.layer_operands(T, E, topk, H, I, T + H)
    y = X.layer(x, logits, topk, *w)
    ids = X.R.choose(logits, topk)[0]

    def differs(x=x, w=w, ids=ids):
        return (X.layer(x, logits, topk, *w, ids=ids) != y).mean(1).min()   # of the least token
    assert (y != 0).mean(1).min() > 0.9
    for block in {0, H // 64, H // 32 - 1}:             # a block of H, where x is not its only one
        less = x.copy()
        less[:, 32 * block:32 * block + 32] = 0
        assert differs(x=less) > 0.5, block
    for first in {I - 32, 0}:                           # a block of I
        w2 = w[2].copy()
        w2[:, :, first // 2:first // 2 + 16] = 0
        assert differs(w=(w[0], w[1], w2, w[3])) > 0.5, first
    gone = ids.copy()                                   # a place
    gone[:, (ids >= 0).sum(1).min() - 1] = -1
    assert differs(ids=gone) > 0.5
    other = w[3].copy()                                 # the scale of the last block
    other[:, :, -1] ^= 127 ^ 128
    assert differs(w=(w[0], w[1], w[2], other)) > 0.5


def test_bf16_rounds_to_nearest_even():
    import torch
    v = np.concatenate((np.arange(-70000, 70000) / 4.0, [0.0, -0.0]))
    want = torch.from_numpy(v).to(torch.float32).to(torch.bfloat16).double().numpy()
    assert np.array_equal(X.bf16(v), want)
