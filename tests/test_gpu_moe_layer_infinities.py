"""Infinities in the mixture-of-experts layer: a sum that holds an infinity of one
sign is that infinity, whatever lies behind the row's end.

Operands are built so that the answer follows from signs alone: gate and up
weights are positive, the rows of W2 have one sign each, so an infinity in x or
among the activated values reaches y[t][h] with the sign of row h."""
import numpy as np
import pytest

from tests import mx_ref as R
from tests.gpu_util import dev, require_gpu, torch_mod

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def wob():
    require_gpu()
    import weight_only_bit_amd as w
    w.device_check()
    return w


def _bytes(codes):
    return (codes[..., 0::2] | codes[..., 1::2] << 4).astype(np.uint8)


def _inputs(T, E, H, I, seed):
    """x, logits, weights and the signs of W2's rows; no code is a zero."""
    torch = torch_mod()
    rng = np.random.default_rng(seed)
    x = torch.from_numpy(rng.uniform(0.5, 1.5, (T, H)).astype(np.float32)).to(torch.bfloat16)
    logits = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32))
    negative = np.broadcast_to(rng.integers(0, 2, (H, 1)), (E, H, 1))  # the same in every expert
    w1 = _bytes(rng.integers(1, 8, (E, 2 * I, H)))
    w2 = _bytes(rng.integers(1, 8, (E, H, I)) + 8 * negative)
    w1s = rng.integers(112, 115, (E, 2 * I, H // 32), np.uint8)
    w2s = rng.integers(112, 115, (E, H, I // 32), np.uint8)
    return x, logits, [w1, w1s, w2, w2s], np.where(negative[0, :, 0] == 1, -np.inf, np.inf)


def _layer(wob, x, logits, topk, w):
    return wob.mxfp4_moe_layer(x.cuda(), logits.cuda(), topk, *(dev(a) for a in w)).double().cpu().numpy()


SHAPES = [(640, 640), (1152, 384), (384, 2176), (192, 320), (2048, 128)]
# beyond 64 tokens rows of whole spans of 128 only: the stages' last span multiplies zeros with what it finds
CASES = [(T, H, I) for T in (1, 2, 5, 8, 9, 33, 66) for H, I in SHAPES if T <= 64 or (H | I) % 128 == 0]


@pytest.mark.parametrize("T,H,I", CASES)
def test_infinity_in_x(wob, T, H, I):
    """In the last block of a token's row: that token's outputs are infinities, the others
    are what they are without it."""
    x, logits, w, want = _inputs(T, 4, H, I, T + H)
    clean = _layer(wob, x, logits, 2, w)
    t = T - 1
    x[t, H - 3] = float("inf")
    y = _layer(wob, x, logits, 2, w)
    assert np.array_equal(y[t], want)
    assert np.isfinite(clean).all() and np.array_equal(y[:t], clean[:t])


@pytest.mark.parametrize("T,H,I", CASES)
def test_activated_value_past_the_range(wob, T, H, I):
    """The last activated value alone is past bf16's and binary32's range."""
    x, logits, w, want = _inputs(T, 4, H, I, T + I)
    w[1][:, I - 1], w[1][:, 2 * I - 1] = 220, 220   # gate and up of about H 2^93
    y = _layer(wob, x, logits, 2, w)
    assert np.array_equal(y, np.broadcast_to(want, y.shape))


@pytest.mark.parametrize("T", [1, 8, 9, 33])
def test_finite_rows_of_one_sign(wob, T):
    """The same operands without an infinity, against the 64-bit reference."""
    x, logits, w, _ = _inputs(T, 4, 640, 640, T)
    y = _layer(wob, x, logits, 2, w)
    ids, p, _ = R.choose(logits.numpy(), 2)
    ref, bound = R.layer(x.double().numpy(), ids, p, *w)
    assert (np.abs(y - ref) <= R.rounded(ref, bound, "bf16")).all()
