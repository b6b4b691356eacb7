"""Scores of the group-limited choice next to a rounding border of binary32, where the 64-bit
score's own error decides."""
import decimal

import numpy as np
import pytest

from tests.gpu_util import require_gpu, torch_mod

pytestmark = pytest.mark.gpu

# (l, top) in hexadecimal, with a difference of -46 to -86.  exp(l - top) lies 2^-49.5 to 2^-46.3 of its
# value from the middle between two binary32 numbers, and on the other side of it once the
# exponential's argument (l - top) * log2 e is rounded to 64 bits (the first six), or the difference, too.
PAIRS = [
    ("-0x1.9e162ap+5", "0x1.0953a2p+0"), ("-0x1.e46dd6p+5", "0x1.13ae52p+0"), ("-0x1.e33084p+5", "0x1.3b5892p+0"),
    ("-0x1.34ac4ap+6", "0x1.daf954p+0"), ("-0x1.9c97a8p+5", "0x1.3923e2p+0"), ("-0x1.017792p+6", "0x1.0d5fc4p+0"),
    ("-0x1.10544cp+6", "0x1.330962p-28"), ("-0x1.33b1c8p+6", "0x1.a149p-31"), ("-0x1.41c98p+6", "0x1.b954f8p-31"),
    ("-0x1.4ce738p+6", "0x1.0f4f18p-29"), ("-0x1.e12036p+5", "0x1.30fddp-25"), ("-0x1.48d34ep+6", "0x1.885d82p-32"),
    ("-0x1.38bd84p+6", "0x1.93c98ap-24"), ("-0x1.40669ap+6", "0x1.bb2cfp-31"), ("-0x1.3ecf4p+6", "0x1.f7453cp-28"),
    ("-0x1.483b7ep+6", "0x1.66e1dap-32"), ("-0x1.1bd7a6p+6", "0x1.151628p-29"), ("-0x1.be3124p+5", "0x1.69058cp-32"),
    ("-0x1.d0198p+5", "0x1.60025ap-31"), ("-0x1.2517e2p+6", "0x1.f12a5p-30"),
]


@pytest.fixture(scope="module")
def wob():
    require_gpu()
    import weight_only_bit_amd as w
    w.device_check()
    return w


def nearest(d):
    """The binary32 number nearest to a Decimal."""
    near = np.float32(float(d))
    around = [np.nextafter(near, np.float32(0)), near, np.nextafter(near, np.float32(np.inf))]
    return min(around, key=lambda f: abs(decimal.Decimal(float(f)) - d))


def scores(wob, logits, score, T):
    """Every expert's score, in the experts' order, for T copies of the rows (the forms differ with T)."""
    torch = torch_mod()
    rows, E = logits.shape
    l = logits.repeat(-(-T // rows), 1).cuda()
    ids, w = wob.moe_route(l, E, score=score, renormalize=False)
    got = torch.zeros_like(w).scatter_(1, ids.long(), w).cpu().numpy()
    assert all(np.array_equal(got[:rows], got[i:i + rows][:rows]) for i in range(0, got.shape[0] - rows + 1, rows))
    return got[:rows]


@pytest.mark.parametrize("T", (1, 4096))
@pytest.mark.parametrize("E", (2, 64))
def test_softmax_next_to_a_rounding_border(wob, E, T):
    """The sum is 1 up to 2^-58, so the score is the exponential."""
    torch = torch_mod()
    pairs = np.array([[float.fromhex(a), float.fromhex(b)] for a, b in PAIRS])
    assert (pairs == pairs.astype(np.float32)).all()
    logits = torch.full((len(PAIRS), E), -700.0)
    logits[:, E - 2:] = torch.from_numpy(pairs).float()
    got = scores(wob, logits, wob.SCORE_SOFTMAX, T)
    with decimal.localcontext() as ctx:
        ctx.prec = 50
        p = [(decimal.Decimal(a) - decimal.Decimal(b)).exp() for a, b in pairs]
        want = np.array([nearest(e / (1 + e)) for e in p])
    assert np.array_equal(got[:, E - 2], want), np.nonzero(got[:, E - 2] != want)
    assert (got[:, E - 1] == 1).all() and (got[:, :E - 2] == 0).all()


def test_sigmoid_of_large_negative_logits(wob):
    """Rounded correctly but for one value in 2^23, as for small logits."""
    torch = torch_mod()
    g = torch.Generator().manual_seed(3)
    logits = -20.0 - 67.0 * torch.rand((1 << 14, 64), generator=g)
    got = scores(wob, logits, wob.SCORE_SIGMOID, 1)
    l = logits.numpy().astype(np.longdouble)
    assert np.finfo(np.longdouble).nmant >= 63  # x86
    want = (1 / (1 + np.exp(-l))).astype(np.float32)
    assert (got != want).sum() <= 1


@pytest.mark.parametrize("score", (0, 1))
def test_extreme_logits(wob, score):
    """Largest and smallest finite logits, infinities and differences past the exponent's range."""
    torch = torch_mod()
    big = torch.finfo(torch.float32).max
    inf = float("inf")
    rows = torch.tensor([[big, -big, 0.0, 1.0], [-big, -big, -big, -big / 2], [inf, big, -inf, inf], [big, big, 1e30, -inf],
                         [-inf, -inf, -inf, -3.0], [1e-45, 0.0, -1e-45, 700.0], [-87.0, -104.5, -110.0, 0.0]])
    T = rows.shape[0]
    ids, w = wob.moe_route(rows.cuda(), 4, score=score, renormalize=False)
    got = torch.zeros((T, 5)).scatter_(1, torch.where(ids < 0, 4, ids).long().cpu(), w.cpu())[:, :4].numpy()
    l = rows.double().numpy()
    with np.errstate(all="ignore"):
        if score == wob.SCORE_SIGMOID:
            want = 1 / (1 + np.exp(-l))
        else:
            top = l.max(-1, keepdims=True)
            e = np.where(l == top, 1.0, np.exp(l - top))
            want = e / e.sum(-1, keepdims=True)
    want = np.where(l == -np.inf, 0, want).astype(np.float32)
    assert np.array_equal(got, want)
    assert np.array_equal((ids.cpu().numpy() < 0).sum(-1), (l == -np.inf).sum(-1))
