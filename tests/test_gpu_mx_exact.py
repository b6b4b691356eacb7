"""The MXFP4 product and the mixture-of-experts layer on operands whose results are exact
(mx_exact.py): every output equals the reference's, at every form of every kernel and on
both sides of every limit."""
import numpy as np
import pytest

from tests import mx_exact as X
from tests.gpu_util import dev, require_gpu, torch_mod
from tests.test_kernel_forms import FEW, TILES

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def wob():
    require_gpu()
    import weight_only_bit_amd as w
    w.device_check()
    return w


def _check_product(wob, M, N, K):
    torch = torch_mod()
    ops = X.product_operands(M, N, K, M + N + K)
    want = X.product(*ops)
    on = [dev(o) for o in ops]
    # bytes of every bit on entry, and none after the end is written
    need = wob.mxfp4_gemm_workspace_size(M, N, K)
    work = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    for dtype in (torch.float32, torch.bfloat16):
        buf = torch.full((M + 2, N), float("nan"), dtype=dtype, device="cuda")
        wob.mxfp4_gemm(*on, out=buf[1:M + 1], workspace=work[:need] if need else None)
        y = buf[1:-1].double().cpu().numpy()
        wrong = np.argwhere(y != (want if dtype == torch.float32 else X.bf16(want)))
        assert len(wrong) == 0, (len(wrong), wrong[:4], dtype)
        assert torch.isnan(buf[0]).all() and torch.isnan(buf[-1]).all(), "write outside y"
    assert (work[need:] == 0xFF).all(), "write past the workspace"


@pytest.mark.parametrize("M,N,K", sorted(TILES.values()))
def test_product_every_tile(wob, M, N, K):
    _check_product(wob, M, N, K)


@pytest.mark.parametrize("M", [17, 64])
@pytest.mark.parametrize("K", [453664, 475168])
def test_product_longest_rows_of_the_64_x_64_tile(wob, M, K):
    """56 spans a part, the most whose scales are loaded at the start, and 59, which are packed."""
    _check_product(wob, M, 72, K)


@pytest.mark.parametrize("M,N,K", [(1000, 2104, 8160), (1000, 2104, 8224), (65, 72, 86048), (65, 72, 90144),
                                   (128, 200, 90112), (100, 5376, 21504), (100, 264, 5632), (100, 264, 5664)])
def test_product_parts_of_the_128_row_tiles(wob, M, N, K):
    """Spans of a part: 16 and 17 (scales of the 128 x 128 tile loaded and packed), 11 and 12."""
    _check_product(wob, M, N, K)


@pytest.mark.parametrize("M,N,K", [
    (16, 72, 8608), (16, 72, 8640), (17, 72, 8608), (15, 40, 9152), (8, 40, 16384), (1, 40, 53248), (1, 40, 53600),
    (1, 24, 65536), (2, 24, 65568), (1, 8, 131072), (1, 4088, 4064), (1, 4096, 64), (2, 4104, 4128), (1, 200, 4096),
    (1, 64, 21504), (3, 5376, 21504), (64, 128, 21504), (130, 256, 21536), (13, 5760, 2880)])
def test_product_few_rows_and_long_rows(wob, M, N, K):
    _check_product(wob, M, N, K)


@pytest.mark.parametrize("M,N", [(1, 24), (16, 24), (33, 72), (100, 72), (1000, 2104)])
@pytest.mark.parametrize("K", [32, 64, 96, 128, 160, 480, 512, 544, 1024, 1056, 1504])
def test_product_ragged_spans(wob, M, N, K):
    _check_product(wob, M, N, K)


@pytest.mark.parametrize("K", [32, 160, 512, 992, 2080])
def test_product_largest_tile(wob, K):
    _check_product(wob, 2050, 4360, K)


def _check_layer(wob, T, E, topk, H, I):
    torch = torch_mod()
    x, logits, w = X.layer_operands(T, E, topk, H, I, T + E + topk + H)
    want = X.layer(x, logits, topk, *w)
    need = wob.moe_layer_workspace_size(T, topk, E, H, I)
    work = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    out = torch.full((T + 2, H), float("nan"), dtype=torch.bfloat16, device="cuda")
    wob.mxfp4_moe_layer(torch.from_numpy(x).to(torch.bfloat16).cuda(), dev(logits), topk, *(dev(a) for a in w),
                        out=out[1:T + 1], workspace=work[:need])
    y = out[1:-1].double().cpu().numpy()
    wrong = np.argwhere(y != want)
    assert len(wrong) == 0, (len(wrong), wrong[:4])
    assert torch.isnan(out[0]).all() and torch.isnan(out[-1]).all(), "write outside y"
    assert (work[need:] == 0xFF).all(), "write past the workspace"


@pytest.mark.parametrize("T,E,topk,H,I", sorted(FEW.values()))
def test_layer_every_form(wob, T, E, topk, H, I):
    _check_layer(wob, T, E, topk, H, I)


@pytest.mark.parametrize("T", [1, 4, 5, 8, 9, 16, 33, 64, 70])
def test_layer_2880(wob, T):
    """Rows that end in half a step, with few experts and four places."""
    _check_layer(wob, T, 8, 4, 2880, 2880)


@pytest.mark.parametrize("T,E,topk,H,I", [
    (64, 16, 8, 128, 64), (65, 16, 8, 128, 64), (64, 16, 9, 128, 64), (8, 70, 64, 64, 64), (9, 70, 64, 64, 64),
    (57, 33, 9, 192, 64), (5, 256, 6, 64, 128), (5, 257, 6, 64, 128), (1, 256, 64, 64, 64),
    (1, 3, 2, 4160, 64), (3, 3, 2, 8192, 64), (9, 2, 1, 6208, 192), (1, 3, 2, 64, 4160), (3, 3, 2, 64, 8192),
    (9, 2, 1, 192, 6208), (8, 2, 2, 8448, 64), (8, 2, 2, 8512, 64), (8, 2, 2, 64, 8960), (8, 2, 2, 64, 9024),
    (1, 4, 4, 64, 4096), (1, 70, 34, 128, 1792), (1, 70, 35, 128, 1792), (4, 40, 34, 128, 1792),
    (4, 40, 35, 128, 1792), (4, 9, 3, 128, 2112), (5, 9, 3, 128, 2112), (8, 9, 3, 128, 2048), (9, 9, 3, 128, 2048),
    (3, 5, 2, 2048, 2112), (12, 5, 2, 1024, 1088), (1, 2, 2, 64, 32768), (1, 2, 2, 32768, 64), (1, 2, 2, 32832, 64),
    (1, 2, 1, 64, 32768), (1, 2, 1, 64, 32832)])
def test_layer_at_the_limits_of_its_kernels(wob, T, E, topk, H, I):
    _check_layer(wob, T, E, topk, H, I)


@pytest.mark.parametrize("T", [2, 8, 9, 40, 66])
@pytest.mark.parametrize("H,I", [(64, 64), (128, 192), (320, 128), (704, 1216), (1152, 640)])
def test_layer_ragged_steps(wob, T, H, I):
    _check_layer(wob, T, 5, 2, H, I)


@pytest.mark.parametrize("T,E,topk,H,I", [
    (64, 4, 4, 128, 192), (32, 8, 8, 192, 128), (33, 8, 8, 192, 128), (40, 32, 8, 128, 64), (41, 32, 8, 128, 64),
    (64, 64, 8, 128, 64), (64, 16, 8, 576, 448), (48, 8, 2, 4096, 64), (49, 8, 2, 4096, 64), (48, 8, 2, 64, 7168),
    (49, 8, 2, 64, 7168), (64, 64, 4, 4096, 128), (33, 64, 8, 4096, 64), (8, 8, 8, 7168, 128)])
def test_layer_at_the_limits_of_pairs(wob, T, E, topk, H, I):
    _check_layer(wob, T, E, topk, H, I)


@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (1, 4104, 4096), (1, 4104, 4064), (8, 4112, 2880), (9, 4112, 2880),
                                   (9, 4096, 2880), (9, 4112, 2048), (9, 4112, 2080), (16, 4104, 8192),
                                   (16, 4096, 8192), (2, 8200, 1056)])
def test_product_few_rows_workgroup_shapes(wob, M, N, K):
    """One and two groups of rows a workgroup, eight and four waves a group."""
    _check_product(wob, M, N, K)


@pytest.mark.parametrize("M,N,K", [(2048, 8704, 96), (2048, 4096, 96), (1030, 14000, 96), (1030, 14000, 640),
                                   (300, 16384, 224), (300, 16392, 224), (128, 16384, 96), (128, 16400, 128),
                                   (250, 8192, 96), (250, 8256, 96), (64, 16384, 96), (65, 16384, 96)])
def test_product_on_both_sides_of_the_tiles_limits(wob, M, N, K):
    """By rounds of 256 x 256 and 128 x 128 tiles, by the number of small and middle tiles, by rows."""
    _check_product(wob, M, N, K)
