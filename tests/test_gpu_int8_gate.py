"""The gate of the 8-bit rows, silu(g) * u in binary32, over the whole range of g.  Every value of
a row is the same, so the row's scale is that value / 127 and shows each bit of it."""
import numpy as np
import pytest

from tests.gpu_util import require_gpu, torch_mod
from tests.test_gpu_int8 import _dt

pytestmark = pytest.mark.gpu

# In half steps of binary32, 2^-24: the exponential and the reciprocal are off by a step each at most (2 and
# 2), the exponential's correction, itself below 2^-17, by a half, and the corrected exponential, the sum 1 + e, the
# products with g and u and the scale's division by 127 round (5).
BOUND = 9.5 * 2.0 ** -24 * 1.001


@pytest.fixture(scope="module")
def wob():
    require_gpu()
    import weight_only_bit_amd as w
    w.device_check()
    return w


def scales(wob, g, u, K):
    """Scales of rows whose K gates are g and whose K ups are u."""
    torch = torch_mod()
    x = torch.cat((g[:, None].expand(-1, K), u[:, None].expand(-1, K)), 1).contiguous().cuda()
    codes, s = wob.int8_quantize(x, act=wob.ACT_SILU_MUL)
    return codes.cpu().numpy(), s.cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("dtype", ("fp32", "bf16", "fp16"))
@pytest.mark.parametrize("lo,hi", [(-88.7, -87.0), (-88.0, -60.0), (-60.0, -20.0), (-20.0, 0.0), (0.0, 20.0), (20.0, 300.0)])
def test_every_gate(wob, dtype, lo, hi):
    """e^-g is finite above -88.72; the ups bring small values up to where a scale is no subnormal."""
    torch = torch_mod()
    n = 8192
    g = (lo + (hi - lo) * torch.rand(n, generator=torch.Generator().manual_seed(7), dtype=torch.float64)).to(_dt(dtype))
    g = g[(g.double() > -88.72) & (g != 0)]
    gd = g.double().numpy()
    silu = gd / (1.0 + np.exp(-gd))
    most = {"fp32": 126, "bf16": 126, "fp16": 15}[dtype]
    u = torch.from_numpy(np.exp2(np.clip(np.round(-np.log2(np.abs(silu))), -14, most))).to(_dt(dtype))
    want = np.abs(silu * u.double().numpy())
    assert (want / 127 > 2.0 ** -126).all()
    for K in (16, 528):
        codes, s = scales(wob, g, u, K)
        off = np.abs(s * 127 - want) / want
        worst = off.argmax()
        assert off[worst] <= BOUND, (gd[worst], np.log2(off[worst]))
        assert (codes == np.where(silu < 0, -127, 127)[:, None]).all()


def test_gates_past_the_exponential(wob):
    """Where e^-g passes binary32 the quotient is a zero, and large gates are themselves."""
    torch = torch_mod()
    g = torch.tensor([-89.0, -100.0, -1e4, -3e38, -0.0, 0.0, 3e38, 2.0 ** 100, 2.0 ** -100, -(2.0 ** -100)])
    u = torch.tensor([1e38, 1e38, 3e38, 3e38, 3e38, 3e38, 1.0, 2.0, 4.0, 4.0])
    codes, s = scales(wob, g, u, 16)
    assert (s[:6] == 0).all() and (codes[:6] == 0).all()
    want = np.array([float(g[6]), 2.0 ** 101, 2.0 ** -99, 2.0 ** -99]).astype(np.float32) / np.float32(127)
    assert (np.abs(s[6:] - want) <= BOUND * want).all() and (np.abs(codes[6:]) == 127).all()


@pytest.mark.parametrize("dtype", ("fp32", "bf16", "fp16"))
def test_gates_that_are_not_finite(wob, dtype):
    """An infinite gate or a NaN, whatever the up value: the row reads back as NaN, its neighbours do not."""
    torch = torch_mod()
    x = torch.ones((7, 2 * 528), dtype=_dt(dtype), device="cuda")
    x[1, 5], x[3, 527], x[5, 0] = float("inf"), float("-inf"), float("nan")
    x[5, 528] = 0
    codes, s = wob.int8_quantize(x, act=wob.ACT_SILU_MUL)
    assert torch.isnan(s).tolist() == [False, True, False, True, False, True, False]
    assert (codes[1::2] == 0).all() and (codes[::2] == 127).all()
