"""GPU parity of the MXFP4 quantisation and the MXFP4 x MXFP4 product against
the 64-bit references of mx_ref.py, through the binding.

Quantisation: exact, byte for byte.  Product: within the bound that mx_ref
derives from K fp32 additions and one rounding of the output.  Guard rows
around every output catch writes outside it.
"""
import numpy as np
import pytest

from tests import mx_ref as R
from tests.gpu_util import dev, require_gpu, torch_mod

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


def _quantize_checked(wob, x):
    """wob.mxfp4_quantize with guard bytes around both outputs, checked exactly."""
    torch = torch_mod()
    rows, K = x.shape
    c = torch.full((rows + 2, K // 2), 0x5A, dtype=torch.uint8, device="cuda")
    # 16 guard bytes in front keep the scale pointer aligned
    s = torch.full((rows * (K // 32) + 32,), 0x5A, dtype=torch.uint8, device="cuda")
    sv = s[16:16 + rows * (K // 32)].view(rows, K // 32)
    wob.mxfp4_quantize(x, out=c[1:rows + 1], out_scale=sv)
    torch.cuda.synchronize()
    assert (c[0] == 0x5A).all() and (c[-1] == 0x5A).all()
    assert (s[:16] == 0x5A).all() and (s[16 + rows * (K // 32):] == 0x5A).all()
    codes, scale = R.quantize(x.double().cpu().numpy())
    assert np.array_equal(sv.cpu().numpy(), scale)
    got = c[1:rows + 1].cpu().numpy()
    assert np.array_equal(got, codes), np.argwhere(got != codes)[:5]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,K", [(1, 32), (1, 5376), (3, 64), (7, 96), (33, 2880), (257, 160),
                                    (64, 1024), (1000, 32)])
def test_quantize_random(wob, dtype, rows, K):
    torch = torch_mod()
    g = torch.Generator().manual_seed(rows * K)
    x = torch.randn((rows, K), generator=g) * torch.exp2(
        torch.randint(-12, 8, (rows, 1), generator=g).float())
    _quantize_checked(wob, x.to(_dt(dtype)).cuda())


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_quantize_every_16_bit_value(wob, dtype):
    """Every bit pattern, each as the largest of its block and beside larger ones."""
    torch = torch_mod()
    v = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(_dt(dtype))
    alone = torch.zeros((65536, 32), dtype=_dt(dtype))
    alone[:, 5] = v
    _quantize_checked(wob, alone.cuda())
    finite = v[torch.isfinite(v.float())]
    n = finite.numel() // 31
    for top in (6.0, 7.5, 1.0, 0.011, 1000.0):
        m = torch.full((n + 1, 32), top, dtype=_dt(dtype))
        vals = torch.clamp(finite.float(), -top, top).to(_dt(dtype))
        m[:n, 1:] = vals[:n * 31].view(n, 31)
        m[n, 1:1 + vals.numel() - n * 31] = vals[n * 31:]
        _quantize_checked(wob, m.cuda())


def test_quantize_fp32_edges(wob):
    """Ties, their neighbours in the last place and the ends of the exponent range, at
    every scale."""
    torch = torch_mod()
    q = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0], np.float32)
    near = np.concatenate((q, np.nextafter(q, np.float32(0)), np.nextafter(q, np.float32(9)), [0.0]))
    block = np.zeros((256, 32), np.float32)
    X = np.arange(-130, 126)
    block[:, :28] = np.ldexp(near.astype(np.float64), X[:, None]).astype(np.float32)
    block[:, 28] = np.ldexp(4.0, X)       # amax in [4, 8) 2^X
    block[:, 29] = -block[:, 0]
    block[:, 30] = -0.0
    block[:, 31] = np.ldexp(-7.9999, X).astype(np.float32)
    _quantize_checked(wob, torch.from_numpy(block).cuda())
    sub = np.zeros((24, 64), np.float32)  # subnormals
    sub[np.arange(24), 3] = np.ldexp(1.0, np.arange(-149, -125)).astype(np.float32)
    sub[:, 40] = np.float32(2.0 ** -128)
    sub[:, 41] = np.float32(3 * 2.0 ** -129)
    _quantize_checked(wob, torch.from_numpy(sub).cuda())


@pytest.mark.parametrize("dtype", DTYPES)
def test_quantize_nan_and_infinity_blocks(wob, dtype):
    torch = torch_mod()
    x = torch.randn((4, 128), generator=torch.Generator().manual_seed(0))
    x[0, 3], x[1, 64], x[2, 127], x[3, 32] = float("nan"), float("inf"), -float("inf"), -float("nan")
    x[3, 40] = float("inf")
    _quantize_checked(wob, x.to(_dt(dtype)).cuda())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,K,width,first", [(5, 64, 72, 0), (33, 2880, 5760, 2880), (1, 96, 104, 8),
                                                (130, 32, 4096, 64)])
def test_quantize_column_slice(wob, dtype, rows, K, width, first):
    torch = torch_mod()
    wide = torch.randn((rows, width), generator=torch.Generator().manual_seed(K)).to(_dt(dtype)).cuda()
    x = wide[:, first:first + K]
    assert rows == 1 or not x.is_contiguous()
    _quantize_checked(wob, x)


def test_quantize_leading_dimensions_and_empty(wob):
    torch = torch_mod()
    x = torch.randn((3, 5, 64), generator=torch.Generator().manual_seed(4)).cuda()
    c, s = wob.mxfp4_quantize(x)
    c2, s2 = wob.mxfp4_quantize(x.view(15, 64))
    assert c.shape == (3, 5, 32) and s.shape == (3, 5, 2)
    assert torch.equal(c.view(15, 32), c2) and torch.equal(s.view(15, 2), s2)
    c, s = wob.mxfp4_quantize(torch.empty((0, 64), device="cuda"))
    assert c.shape == (0, 32) and s.shape == (0, 2)
    c, s = wob.mxfp4_quantize(x[0, 0])
    assert torch.equal(c, c2[0]) and torch.equal(s, s2[0])


def test_quantize_refuses_unaligned_rows(wob):
    torch = torch_mod()
    wide = torch.zeros((4, 70), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        wob.mxfp4_quantize(wide[:, :64])       # rows 140 bytes apart
    with pytest.raises(ValueError):
        wob.mxfp4_quantize(torch.zeros((4, 72), dtype=torch.bfloat16, device="cuda")[:, 4:68])


# ---- product ---------------------------------------------------------------

def _operands(M, N, K, seed, lo=118, hi=126):
    rng = np.random.default_rng(seed)
    return (rng.integers(0, 256, (M, K // 2), np.uint8), rng.integers(lo, hi + 1, (M, K // 32), np.uint8),
            rng.integers(0, 256, (N, K // 2), np.uint8), rng.integers(lo, hi + 1, (N, K // 32), np.uint8))


def _product(wob, ops, out):
    """wob.mxfp4_gemm into guarded rows -> float64 [M, N]."""
    torch = torch_mod()
    x, xs, w, ws = ops
    M, N = x.shape[0], w.shape[0]
    buf = torch.full((M + 2, N), float("nan"), dtype=_dt(out), device="cuda")
    # a row of N elements keeps the 16-byte alignment where N % 8 == 0
    wob.mxfp4_gemm(dev(x), dev(xs), dev(w), dev(ws), out=buf[1:M + 1])
    torch.cuda.synchronize()
    assert torch.isnan(buf[0]).all() and torch.isnan(buf[-1]).all(), "write outside y"
    return buf[1:-1].double().cpu().numpy()


def _check(wob, ops, out):
    y = _product(wob, ops, out)
    ref, bound = R.product(*ops)
    off = np.abs(y - ref)
    tol = R.rounded(ref, bound, out)
    assert (off <= tol).all(), (np.argwhere(~(off <= tol))[:4], float((off / tol).max()))


@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65])
@pytest.mark.parametrize("N,K", [(8, 32), (16, 64), (40, 96), (72, 352), (264, 512), (520, 1152)])
def test_product_small(wob, M, N, K):
    _check(wob, _operands(M, N, K, M * N + K), "fp32")


@pytest.mark.parametrize("M", [100, 127, 128, 129, 192, 255, 256, 257, 300, 520])
@pytest.mark.parametrize("N,K", [(8, 64), (256, 128), (136, 288), (512, 1024), (776, 2912)])
def test_product_larger(wob, M, N, K):
    _check(wob, _operands(M, N, K, M + N + K), "fp32")


@pytest.mark.parametrize("out", DTYPES)
@pytest.mark.parametrize("M,N,K", [(1, 2880, 2880), (4, 512, 5376), (16, 1000, 672), (96, 5760, 2880),
                                   (333, 640, 2880)])
def test_product_output_types(wob, out, M, N, K):
    ops = _operands(M, N, K, N + K, 117, 121)
    _check(wob, ops, out)


@pytest.mark.parametrize("M,N,K", [(1, 64, 21504), (3, 5376, 21504), (64, 128, 21504), (130, 256, 21536)])
def test_product_long_rows(wob, M, N, K):
    _check(wob, _operands(M, N, K, 3, 120, 123), "fp32")


@pytest.mark.parametrize("M,N,K", [(1000, 1096, 6144), (1000, 1096, 6240), (1000, 1032, 6560),
                                   (1100, 2040, 6176), (70, 9224, 6336), (127, 5000, 12288),
                                   (1100, 2040, 512), (1400, 2048, 640), (260, 8200, 352),
                                   (1030, 8192, 480), (20, 16392, 14880), (20, 16392, 14496),
                                   (1000, 2104, 8160), (1000, 2104, 8224), (70, 9224, 8160),
                                   (1030, 14000, 96), (2048, 8704, 64), (300, 16384, 224)])
def test_product_many_rows_long(wob, M, N, K):
    """Too few tiles for the largest one, and rows too long or too many for the smallest."""
    _check(wob, _operands(M, N, K, 5, 117, 121), "fp32")


@pytest.mark.parametrize("M", [17, 33, 64, 65])
@pytest.mark.parametrize("N,K", [(72, 5376), (2056, 6240), (16392, 1056), (72, 453664), (72, 475168)])
def test_product_narrow(wob, M, N, K):
    """17 to 64 rows: whole and in parts, scales from the rows, loaded at the start, packed."""
    _check(wob, _operands(M, N, K, K + M, 117, 121), "fp32")


@pytest.mark.parametrize("K", [32, 96, 128, 480, 512, 544, 992, 1056, 2080])
def test_product_largest_tile(wob, K):
    """Ragged in rows, columns and spans."""
    _check(wob, _operands(2050, 4360, K, K, 117, 121), "fp32")


@pytest.mark.parametrize("out", DTYPES)
def test_product_largest_tile_output_types(wob, out):
    _check(wob, _operands(2045, 4360, 160, 3, 117, 121), out)


@pytest.mark.parametrize("M", [1, 5, 40, 140, 300])
def test_product_extreme_scales(wob, M):
    """Scale bytes at both ends whose products are ordinary numbers, and a NaN scale: it
    reaches its whole row or column and nothing else."""
    N, K = 264, 416
    x, xs, w, ws = _operands(M, N, K, M)
    xs[:], ws[:] = 1, 253
    xs[:, 3], ws[:, 3] = 254, 2
    xs[:, 5], ws[:, 5] = 0, 254
    _check(wob, (x, xs, w, ws), "fp32")
    xs[M - 1, 12] = 255
    ws[17, 0] = 255
    y = _product(wob, (x, xs, w, ws), "fp32")
    nan = np.zeros((M, N), bool)
    nan[M - 1], nan[:, 17] = True, True
    assert np.array_equal(np.isnan(y), nan)


@pytest.mark.parametrize("M", [1, 20, 200])
def test_product_overflow_and_zeros(wob, M):
    """Past the output type's range: infinity, as rounding to nearest gives; zero codes: exact zeros."""
    N, K = 64, 256
    x, xs, w, ws = _operands(M, N, K, M)
    x[:], w[:] = 0x66, 0x66                      # every element 4.0
    xs[:], ws[:] = 134, 134                      # 2^7 each: sums of 2^26
    y = _product(wob, (x, xs, w, ws), "fp16")
    assert np.isposinf(y).all()
    w[3:9] = 0x80                                # +0 and -0
    y = _product(wob, (x, xs, w, ws), "fp32")
    assert (y[:, 3:9] == 0).all() and (np.delete(y, range(3, 9), 1) == 2.0 ** 26).all()


def test_product_exact_integers(wob):
    """Whole products below 2^24: fp32 sums are exact whatever their order."""
    for M, N, K in ((1, 512, 1024), (17, 264, 992), (150, 264, 1024), (513, 520, 2912)):
        x, xs, w, ws = _operands(M, N, K, K)
        xs[:], ws[:] = 128, 128                  # every element a whole number up to 12
        y = _product(wob, (x, xs, w, ws), "fp32")
        assert np.array_equal(y, R.product(x, xs, w, ws)[0]), (M, N, K)


@pytest.mark.parametrize("M,N,K", [(1, 16384, 5376), (100, 5376, 21504), (2048, 16384, 5376)])
def test_product_full_size_sampled(wob, M, N, K):
    """Full-size shapes: sampled outputs in every 32 x 128 part against the reference."""
    torch = torch_mod()
    ops = _operands(M, N, K, 5, 117, 121)
    y = wob.mxfp4_gemm(*(dev(o) for o in ops), out_dtype=torch.float32).cpu().numpy()
    assert np.isfinite(y).all()
    rng = np.random.default_rng(6)
    n = np.unique(np.concatenate((np.arange(0, N, 128) + rng.integers(0, 128, (N + 127) // 128), [N - 1])))
    n = n[n < N]
    m = np.unique(np.concatenate((np.arange(0, M, 32) + rng.integers(0, 32, (M + 31) // 32), [M - 1])))
    m = m[m < M]
    x, xs, w, ws = ops
    ref, bound = R.product(x[m], xs[m], w[n], ws[n])
    off = np.abs(y[np.ix_(m, n)] - ref)
    assert (off <= R.rounded(ref, bound, "fp32")).all()


def test_product_repeats_bit_for_bit_and_on_another_stream(wob):
    torch = torch_mod()
    for M, N, K in ((1, 5376, 2880), (48, 1024, 8192), (300, 520, 2912)):
        ops = [dev(o) for o in _operands(M, N, K, 9)]
        first = wob.mxfp4_gemm(*ops)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            again = [wob.mxfp4_gemm(*ops) for _ in range(3)]
        side.synchronize()
        assert all(torch.equal(first, a) for a in again)


def test_product_large_offsets(wob):
    """Codes past 2^31 bytes: rows at the end of a 2.2 GB operand."""
    torch = torch_mod()
    N, K, M = 139264, 32768, 3
    w = torch.zeros((N, K // 2), dtype=torch.uint8, device="cuda")
    ws = torch.full((N, K // 32), 127, dtype=torch.uint8, device="cuda")
    x = torch.full((M, K // 2), 0x22, dtype=torch.uint8, device="cuda")  # ones
    xs = torch.full((M, K // 32), 127, dtype=torch.uint8, device="cuda")
    w[N - 1], w[N - 9], w[7] = 0x22, 0x44, 0x11
    y = wob.mxfp4_gemm(x, xs, w, ws, out_dtype=torch.float32)
    want = torch.zeros((M, N), device="cuda")
    want[:, N - 1], want[:, N - 9], want[:, 7] = K, 2 * K, K / 2
    assert torch.equal(y, want)


def test_quantise_then_product(wob):
    """A dense layer as it is used: weights and activations quantised, then multiplied."""
    torch = torch_mod()
    g = torch.Generator().manual_seed(1)
    x = torch.randn((37, 512), generator=g).to(torch.bfloat16).cuda()
    w = (torch.randn((264, 512), generator=g) * 0.05).cuda()
    xc, xs = wob.mxfp4_quantize(x)
    wc, ws = wob.mxfp4_quantize(w)
    y = wob.mxfp4_gemm(xc, xs, wc, ws, out_dtype=torch.float32).double().cpu().numpy()
    xq, wq = R.quantize(x.double().cpu().numpy()), R.quantize(w.double().cpu().numpy())
    ref, bound = R.product(*xq, *wq)
    assert (np.abs(y - ref) <= R.rounded(ref, bound, "fp32")).all()


@pytest.mark.parametrize("M", [1, 24, 200])
def test_captured_and_replayed(wob, M):
    """Quantise and multiply captured in a graph, replayed over changing inputs with eager
    work between: every replay equals the eager result."""
    torch = torch_mod()
    N, K = 520, 1184
    g = torch.Generator().manual_seed(M)
    w = torch.randn((N, K), generator=g).cuda()
    wc, ws = wob.mxfp4_quantize(w)
    x = torch.randn((M, K), generator=g).cuda()
    work = torch.empty(max(wob.mxfp4_gemm_workspace_size(M, N, K), 16), dtype=torch.uint8, device="cuda")
    xc, xs = wob.mxfp4_quantize(x)
    y = wob.mxfp4_gemm(xc, xs, wc, ws, workspace=work)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        wob.mxfp4_quantize(x, out=xc, out_scale=xs)
        wob.mxfp4_gemm(xc, xs, wc, ws, out=y, workspace=work)
    for k in range(4):
        x.copy_(torch.randn((M, K), generator=g).cuda())
        y.fill_(float("nan"))
        work.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        want = wob.mxfp4_gemm(*wob.mxfp4_quantize(x), wc, ws)
        assert torch.equal(y, want), k


@pytest.mark.parametrize("M,N,K", [
    (16, 72, 8608), (16, 72, 8640), (17, 72, 8608), (15, 40, 9152), (8, 40, 16384),   # rows staged whole
    (1, 40, 53248), (1, 40, 53600), (1, 24, 65536), (2, 24, 65568), (1, 8, 131072),
    (1, 4088, 4064), (1, 4096, 64), (2, 4104, 4128), (1, 200, 4096)])                # workgroup shapes
def test_product_at_the_limits_of_its_kernels(wob, M, N, K):
    """On both sides of the limits of the kernel for few rows."""
    _check(wob, _operands(M, N, K, K + N, 120, 123), "fp32")


@pytest.mark.parametrize("M", [1, 40, 100, 600])
def test_product_on_two_streams_at_once(wob, M):
    """Calls without a common workspace do not disturb each other."""
    torch = torch_mod()
    sets = [[dev(o) for o in _operands(M, 2056, 6240, seed, 117, 121)] for seed in (1, 2)]
    want = [wob.mxfp4_gemm(*s) for s in sets]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in sets], [[], []]
    for _ in range(10):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(wob.mxfp4_gemm(*sets[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(want[i], y) for y in got[i])


def test_quantise_offsets_past_32_bits(wob):
    """More than 2^31 elements, and rows whose distances pass 2^32 bytes."""
    torch = torch_mod()
    K = 16384
    n = (1 << 31) // K + 40
    x = torch.zeros((n, K), dtype=torch.bfloat16, device="cuda")
    rows = [0, 1, n // 2, (1 << 31) // K - 1, (1 << 31) // K, n - 1]
    g = torch.Generator().manual_seed(8)
    v = torch.randn((len(rows), K), generator=g).to(torch.bfloat16)
    x[rows] = v.cuda()
    codes, scale = wob.mxfp4_quantize(x)
    rc, rs = _quant_ref(v)
    assert np.array_equal(codes[rows].cpu().numpy(), rc) and np.array_equal(scale[rows].cpu().numpy(), rs)
    assert not codes[2].any() and not scale[n - 2].any()
    wide = x.view(-1)[:n // 2 * 2 * K].view(-1, 2 * K)[:, 64:64 + 96]   # rows 2 K apart
    codes, scale = wob.mxfp4_quantize(wide)
    wc, wsc = _quant_ref(wide[[0, n // 4, wide.shape[0] - 1]].cpu())
    at = [0, n // 4, wide.shape[0] - 1]
    assert np.array_equal(codes[at].cpu().numpy(), wc) and np.array_equal(scale[at].cpu().numpy(), wsc)


def _quant_ref(v):
    return R.quantize(v.double().numpy())
