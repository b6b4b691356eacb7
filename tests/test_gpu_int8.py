"""GPU parity of the 8-bit rows and their product against block_ref.py, through the
binding.  Without an activation the codes and scales are exact, byte for byte; the product's
32-bit outputs without a bias too, its other outputs within the bound of their roundings.
Guard elements around every output catch writes outside it."""
import numpy as np
import pytest

from tests import block_ref as R
from tests.gpu_util import require_gpu, torch_mod

pytestmark = pytest.mark.gpu

DTYPES = ("bf16", "fp16", "fp32")


@pytest.fixture(scope="module")
def wob():
    require_gpu()
    import weight_only_bit_amd as w
    w.device_check()
    return w


def _dt(name):
    torch = torch_mod()
    return {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[name]


def guarded(shape, dtype, fill):
    """(whole buffer, view of `shape` in its middle): 64 guard elements on both sides."""
    torch = torch_mod()
    n = int(np.prod(shape))
    buf = torch.full((n + 128,), fill, dtype=dtype, device="cuda")
    return buf, buf[64:64 + n].view(shape)


def guards_whole(buf, fill):
    b = buf.float()
    return bool((b[:64] == fill).all() and (b[-64:] == fill).all())


def quantised(wob, x, **kw):
    torch = torch_mod()
    K = x.shape[1] // (2 if kw.get("act") else 1)
    cb, c = guarded((x.shape[0], K), torch.int8, 77)
    sb, s = guarded((x.shape[0],), torch.float32, 77)
    wob.int8_quantize(x, out=c, out_scale=s, **kw)
    torch.cuda.synchronize()
    assert guards_whole(cb, 77) and guards_whole(sb, 77)
    return c.cpu().numpy(), s.cpu().numpy()


def rows(n, K, seed, dtype):
    torch = torch_mod()
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((n, K), generator=g) * torch.exp2(torch.randint(-12, 8, (n, 1), generator=g).float())
    return x.to(_dt(dtype)).cuda()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,K", [(1, 16), (1, 5376), (3, 64), (7, 496), (5, 512), (33, 528), (257, 160),
                                 (6, 2048), (5, 2064), (4, 8192), (3, 8208), (2, 32768), (3, 32784), (2, 65536),
                                 (1000, 32), (300, 2880), (70, 48), (71, 128), (19, 144), (17, 256), (9, 272), (7, 768),
                                 (5, 1024), (6, 1040), (3, 4096), (2, 4112)])
def test_quantize_exact(wob, dtype, n, K):
    x = rows(n, K, n * K, dtype)
    codes, scale = R.int8_rows(x.float().cpu().numpy())
    c, s = quantised(wob, x)
    assert np.array_equal(s, scale)
    assert np.array_equal(c, codes), np.argwhere(c != codes)[:5]


def test_quantize_many_rows(wob):
    """More rows than the grid has workgroups for at once."""
    torch = torch_mod()
    x = (torch.arange(4_200_000, device="cuda") % 251 - 125).to(torch.float32)
    x = (x[:, None] * torch.linspace(-1, 1, 16, device="cuda")).to(torch.bfloat16)
    c, s = wob.int8_quantize(x)
    top = x.float().abs().amax(-1)
    full = torch.full_like(top, 127.0)  # tensor by tensor: torch multiplies by a number's reciprocal
    assert torch.equal(s, torch.div(top, full))
    q = torch.round(x.float() * torch.where(top > 0, torch.div(full, top), 0)[:, None]).to(torch.int8)
    assert torch.equal(c, q)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("K", [64, 2880, 16384])
def test_quantize_special_rows(wob, dtype, K):
    torch = torch_mod()
    x = rows(12, K, K, dtype)
    x[0] = 0
    x[1] = -0.0
    x[2, K - 1] = float("inf")
    x[3, 0] = float("-inf")
    x[4, K // 2] = float("nan")
    x[5] = torch.finfo(x.dtype).max
    x[6] = torch.finfo(x.dtype).smallest_normal * 1.5
    x[7] = 0
    x[7, 3] = torch.finfo(x.dtype).smallest_normal / 4  # a subnormal
    x[8] = 0
    x[8, 5] = -1
    x[9] = torch.arange(K, device="cuda") % 255 - 127  # every code, exact ties none
    x[10] = (torch.arange(K, device="cuda") % 254 - 127) / 2  # half steps once 63.5 is the top
    codes, scale = R.int8_rows(x.float().cpu().numpy())
    c, s = quantised(wob, x)
    assert np.array_equal(s, scale, equal_nan=True)
    assert np.array_equal(c, codes)
    back = wob.int8_dequant(torch.from_numpy(c).cuda(), torch.from_numpy(s).cuda(), out_dtype=torch.float32)
    assert torch.isnan(back[2:5]).all() and not torch.isnan(back[:2]).any()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("K,pad", [(64, 8), (2880, 16), (48, 8), (16384, 1024)])
def test_quantize_column_slice(wob, dtype, K, pad):
    torch = torch_mod()
    wide = rows(9, K + 2 * pad, 5, dtype)
    x = wide[:, pad:pad + K]
    assert not x.is_contiguous()
    codes, scale = R.int8_rows(x.float().cpu().numpy())
    c, s = quantised(wob, x)
    assert np.array_equal(c, codes) and np.array_equal(s, scale)
    c, s = wob.int8_quantize(wide[:1, pad:pad + K])
    assert np.array_equal(c.cpu().numpy(), codes[:1])
    if dtype != "fp32":  # rows that start 8 bytes off a 16-byte border
        with pytest.raises(ValueError):
            wob.int8_quantize(wide[:, 4:4 + K])
    torch.cuda.synchronize()


def test_quantize_leading_dimensions(wob):
    torch = torch_mod()
    x = rows(24, 96, 3, "bf16")
    c, s = wob.int8_quantize(x)
    for lead in ((2, 3, 4), (24, 1), (1, 24)):
        c3, s3 = wob.int8_quantize(x.view(*lead, 96))
        assert c3.shape == (*lead, 96) and s3.shape == lead
        assert torch.equal(c3.view(24, 96), c) and torch.equal(s3.view(24), s)
    c1, s1 = wob.int8_quantize(x[0])
    assert s1.shape == () and torch.equal(c1, c[0]) and s1 == s[0]
    c0, s0 = wob.int8_quantize(x[:0])
    assert c0.shape == (0, 96) and s0.shape == (0,)
    assert torch.equal(wob.int8_dequant(c.view(2, 3, 4, 96), s.view(2, 3, 4)).view(24, 96), wob.int8_dequant(c, s))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,K", [(1, 16), (5, 512), (9, 528), (300, 2880), (3, 8208), (2, 21504), (2, 65536), (37, 64),
                                 (19, 112), (9, 256), (5, 1024)])
def test_quantize_gated(wob, dtype, n, K):
    torch = torch_mod()
    g = torch.Generator().manual_seed(n + K)
    x = (torch.randn((n, 2 * K), generator=g) * 4).to(_dt(dtype)).cuda()
    x[0, :3] = torch.tensor([-200.0, 100.0, -90.0])
    v, dv = R.silu_mul(x.double().cpu().numpy())
    c, s = quantised(wob, x, act=wob.ACT_SILU_MUL)
    top, dtop = np.abs(v).max(-1), dv.max(-1)
    assert (np.abs(s - top / 127) <= (dtop / 127 + top / 127 * 2.0 ** -23)).all()
    # a code stands for the nearest multiple of the scale, up to v's error and the
    # roundings of 127 / amax and of the product (2^-22 of up to 127 steps)
    off = np.abs(c * s.astype(np.float64)[:, None] - v)
    assert (off <= (0.5 + 127 * 3 * 2.0 ** -23) * s[:, None] + dv + dtop[:, None]).all()
    assert np.abs(c.astype(int)).max() == 127


def test_quantize_gated_special(wob):
    torch = torch_mod()
    x = rows(6, 128, 1, "fp32")
    x[0, :64] = 0            # silu(0) = 0
    x[1, 64:] = 0
    x[2, 70] = float("inf")
    x[3, 5] = float("nan")
    x[4, 7], x[4, 71] = 3e38, 3e38   # the product passes binary32's range
    x[5, :64] = -3e38        # silu -> -0
    x[5, 64:] = 1.0
    c, s = quantised(wob, x, act=wob.ACT_SILU_MUL)
    assert (c[[0, 1, 5]] == 0).all() and (s[[0, 1, 5]] == 0).all()
    assert np.isnan(s[2:5]).all() and (c[2:5] == 0).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,K", [(1, 16), (7, 48), (300, 2880), (2, 65536)])
def test_dequant_exact(wob, dtype, n, K):
    torch = torch_mod()
    g = torch.Generator().manual_seed(n)
    c = torch.randint(-128, 128, (n, K), generator=g).to(torch.int8).cuda()
    s = (torch.randn(n, generator=g) * 0.1).cuda()
    buf, out = guarded((n, K), _dt(dtype), 77)
    wob.int8_dequant(c, s, out=out)
    assert torch.equal(out, (c.float() * s[:, None]).to(_dt(dtype))) and guards_whole(buf, 77)


# ---------------------------------------------------------------------------
# The product
# ---------------------------------------------------------------------------

def operands(M, N, K, seed, full=False):
    torch = torch_mod()
    g = torch.Generator().manual_seed(seed)
    lo = -128 if full else -127
    x = torch.randint(lo, 128, (M, K), generator=g).to(torch.int8)
    w = torch.randint(lo, 128, (N, K), generator=g).to(torch.int8)
    xs = torch.exp2(torch.randn(M, generator=g) * 3) * 0.01
    ws = torch.exp2(torch.randn(N, generator=g) * 3) * 0.001
    return x, xs, w, ws, torch.randn(N, generator=g)


def product(wob, x, xs, w, ws, dtype, bias=None):
    torch = torch_mod()
    M, N, K = x.shape[0], w.shape[0], x.shape[1]
    buf, out = guarded((M, N), _dt(dtype), 77)
    need = wob.int8_gemm_workspace_size(M, N, K)
    work = torch.full((max(need, 16),), 0xFF, dtype=torch.uint8, device="cuda")
    wob.int8_gemm(x.cuda(), xs.cuda(), w.cuda(), ws.cuda(), bias=None if bias is None else bias.cuda(),
                  out=out, workspace=work)
    torch.cuda.synchronize()
    assert guards_whole(buf, 77)
    return out.float().cpu().numpy()


SHAPES = [(1, 8, 16), (1, 16, 32), (2, 8, 48), (1, 264, 64), (3, 40, 80), (1, 512, 5376), (4, 264, 2880), (8, 1000, 112),
          (13, 520, 1040), (15, 24, 144), (16, 256, 4096), (16, 136, 21504), (1, 64, 65536), (16, 48, 65552),
          (17, 72, 272), (17, 8, 16), (31, 264, 336), (33, 72, 5376), (48, 128, 8192), (64, 64, 64), (65, 72, 80),
          (70, 520, 2064), (100, 256, 21504), (127, 136, 144), (128, 128, 128), (129, 264, 1040), (200, 1000, 528),
          (255, 520, 16), (256, 256, 272), (257, 264, 400), (300, 2056, 208), (520, 1032, 1088)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product_exact(wob, M, N, K):
    """32-bit outputs without a bias equal the definition operation by operation."""
    x, xs, w, ws, _ = operands(M, N, K, M * 7 + N + K, full=True)
    y = product(wob, x, xs, w, ws, "fp32")
    want = R.product_f32(x.numpy(), xs.numpy(), w.numpy(), ws.numpy())
    assert np.array_equal(y, want), np.argwhere(y != want)[:5]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("bias", (False, True))
@pytest.mark.parametrize("M,N,K", [(1, 264, 2880), (13, 520, 1040), (40, 136, 5376), (100, 264, 4096),
                                   (150, 520, 528), (300, 520, 272)])
def test_product_types(wob, dtype, bias, M, N, K):
    x, xs, w, ws, b = operands(M, N, K, K, full=True)
    y = product(wob, x, xs, w, ws, dtype, b if bias else None)
    want, bound = R.product(x.numpy(), xs.numpy(), w.numpy(), ws.numpy(), b.numpy() if bias else None)
    bound = bound + R.HALF_STEP[dtype] * (np.abs(want) + bound) + R.TINY[dtype]
    if dtype == "fp16":  # from 65520, half a step past its largest value, a rounding gives an infinity
        past = np.abs(want) - bound >= 65520
        assert (y[past] == np.sign(want[past]) * np.inf).all()
        want, y = np.where(past, 0, want), np.where(past, 0, y)
    assert (np.abs(y - want) <= bound).all()


@pytest.mark.parametrize("M", (1, 13, 40, 100, 300))
@pytest.mark.parametrize("K", (16, 1040, 131056))
def test_product_largest_sums(wob, M, K):
    """Every product (-128)^2: the sum reaches 2^31 - 2^18 at the longest row."""
    torch = torch_mod()
    x, w = torch.full((M, K), -128, dtype=torch.int8), torch.full((24, K), -128, dtype=torch.int8)
    y = product(wob, x, torch.ones(M), w, torch.ones(24), "fp32")
    assert (y == np.float32(K * 16384)).all()
    w[1] = 127
    y = product(wob, x, torch.ones(M), w, torch.ones(24), "fp32")
    assert (y[:, 1] == np.float32(-K * 128 * 127)).all() and (y[:, 2] == np.float32(K * 16384)).all()


@pytest.mark.parametrize("M", (1, 16, 40, 100, 300))
def test_product_special_scales(wob, M):
    """NaN and infinite scales stay in their row or column, zero scales give zeros."""
    x, xs, w, ws, b = operands(M, 72, 144, M)
    xs[0] = float("nan")
    ws[3], ws[4], ws[5] = float("nan"), float("inf"), 0.0
    y = product(wob, x, xs, w, ws, "fp32")
    want = R.product_f32(x.numpy(), xs.numpy(), w.numpy(), ws.numpy())
    assert np.array_equal(y, want, equal_nan=True)
    assert np.isnan(y[0]).all() and np.isnan(y[:, 3]).all()
    if M > 1:
        assert np.isfinite(y[1:, 6:]).all() and (y[1:, 5] == 0).all()


def test_product_rows_do_not_depend_on_the_batch(wob):
    """A token's output is the same alone and in any batch (exact sums): every kernel agrees."""
    x, xs, w, ws, b = operands(600, 392, 2896, 9)
    whole = product(wob, x, xs, w, ws, "fp32")
    for M in (1, 2, 8, 9, 16, 17, 33, 64, 65, 100, 129, 256, 257, 513):
        part = product(wob, x[-M:].contiguous(), xs[-M:].contiguous(), w, ws, "fp32")
        assert np.array_equal(part, whole[-M:]), M


def test_product_empty(wob):
    torch = torch_mod()
    x, xs, w, ws, _ = (t.cuda() for t in operands(4, 16, 64, 0))
    assert wob.int8_gemm(x[:0], xs[:0], w, ws).shape == (0, 16)
    assert wob.int8_gemm(x, xs, w[:0], ws[:0]).shape == (4, 0)


def test_offsets_past_31_bits(wob):
    """Operands and outputs whose byte offsets pass 2^31."""
    torch = torch_mod()
    N, K = 65544, 65536  # w: 4295 MB is refused, 32768 rows fewer are 2.1e9 bytes and more
    w = torch.zeros((N, K), dtype=torch.int8, device="cuda")
    xs, ws = torch.ones(3, device="cuda"), torch.ones(N, device="cuda")
    x = torch.ones((3, K), dtype=torch.int8, device="cuda")
    with pytest.raises(ValueError):
        wob.int8_gemm(x, xs, w, ws)
    N = 65528
    w[N - 1, K - 16:] = 1
    w[N - 9, 0] = 5
    for M in (3, 20, 70, 140, 300):
        xm = torch.ones((M, K), dtype=torch.int8, device="cuda")
        y = wob.int8_gemm(xm, torch.ones(M, device="cuda"), w[:N], ws[:N], out_dtype=torch.float32)
        assert (y[:, N - 1] == 16).all() and (y[:, N - 9] == 5).all() and float(y.sum()) == 21 * M
    del w
    M, N = 70000, 16400  # y: 4.6e9 bytes of float32
    x = torch.zeros((M, 16), dtype=torch.int8, device="cuda")
    x[M - 1] = 1
    x[0] = 2
    w = torch.ones((N, 16), dtype=torch.int8, device="cuda")
    y = wob.int8_gemm(x, torch.ones(M, device="cuda"), w, torch.ones(N, device="cuda"), out_dtype=torch.float32)
    assert (y[M - 1] == 16).all() and (y[0] == 32).all() and (y[1:M - 1] == 0).all()
