"""The row operators past the last-level cache, where rows are read in another way, and the
8-bit product of few rows whose weights pass 2^32 bytes less a little: the same rows in small
calls, which the other tests check, give the same bytes."""
import pytest

from tests.gpu_util import require_gpu, torch_mod
from tests.test_gpu_int8 import _dt

pytestmark = pytest.mark.gpu

PAST = 257 << 20  # bytes


@pytest.fixture(scope="module")
def wob():
    require_gpu()
    import weight_only_bit_amd as w
    w.device_check()
    return w


def normal(shape, dtype, seed):
    torch = torch_mod()
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, device="cuda", generator=g).to(_dt(dtype))


def parts(n):
    return (slice(0, 7), slice(n // 2, n // 2 + 7), slice(n - 7, n))


@pytest.mark.parametrize("gated", (False, True))
@pytest.mark.parametrize("dtype", ("bf16", "fp16", "fp32"))
@pytest.mark.parametrize("K", (48, 128, 256, 512, 1024, 2048, 4080, 8192, 16384, 21504, 32768, 65536))
def test_quantise(wob, K, dtype, gated):
    torch = torch_mod()
    act, width = (wob.ACT_SILU_MUL, 2 * K) if gated else (wob.ACT_NONE, K)
    n = PAST // (width * (4 if dtype == "fp32" else 2)) + 3
    x = normal((n, width), dtype, K)
    codes, scale = wob.int8_quantize(x, act=act)
    for at in parts(n):
        c, s = wob.int8_quantize(x[at].clone(), act=act)
        assert torch.equal(codes[at], c) and torch.equal(scale[at], s)
    assert torch.equal(wob.int8_dequant(codes, scale, torch.float32), codes.float() * scale[:, None])


@pytest.mark.parametrize("gate", (None, "channel", "rows"))
@pytest.mark.parametrize("dtype,res", (("bf16", "bf16"), ("fp16", "fp32"), ("fp32", "fp32")))
@pytest.mark.parametrize("H", (64, 128, 256, 512, 1024, 2048, 4064, 8192, 16384, 32768))
def test_norm(wob, H, dtype, res, gate):
    torch = torch_mod()
    n = PAST // (H * ((2 if dtype != "fp32" else 4) + (2 if res != "fp32" else 4))) + 3
    y, r = normal((n, H), dtype, H), normal((n, H), res, H + 1)
    w, post = normal((H,), dtype, 3), normal((H,), dtype, 4)
    g = None if gate is None else normal((H,) if gate == "channel" else (n, H), dtype, 5)
    for quant in (wob.QUANT_NONE, wob.QUANT_INT8, wob.QUANT_MXFP4):
        whole = wob.residual_norm(y, r, w, post_weight=post, gate=g, alpha=0.5, quant=quant)
        for at in parts(n):
            part = wob.residual_norm(y[at].clone(), r[at].clone(), w, post_weight=post, alpha=0.5, quant=quant,
                                     gate=g[at].clone() if gate == "rows" else g)
            for a, b in zip(whole, part):
                assert torch.equal(a[at], b)
    # in place, and without a norm behind the block
    h = wob.residual_norm(y, r.clone(), None, post_weight=post, gate=g, alpha=0.5)[1]
    assert torch.equal(h, whole[-1])
    wob.residual_norm(y, r, w, post_weight=post, gate=g, alpha=0.5, residual_out=r)
    assert torch.equal(h, r)


@pytest.mark.parametrize("M", (1, 2, 5))
def test_few_rows_of_large_weights(wob, M):
    torch = torch_mod()
    N, K = (65528, 65536) if M == 1 else (1 << 19, 8176)
    w = torch.zeros((N, K), dtype=torch.int8, device="cuda")
    w[N - 1, K - 16:] = 1
    w[N - 9, 0] = 5
    x = torch.ones((M, K), dtype=torch.int8, device="cuda")
    y = wob.int8_gemm(x, torch.ones(M, device="cuda"), w, torch.ones(N, device="cuda"), out_dtype=torch.float32)
    assert (y[:, N - 1] == 16).all() and (y[:, N - 9] == 5).all() and float(y.sum()) == 21 * M
