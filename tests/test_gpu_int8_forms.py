"""Every form of the 8-bit product on sizes that take it, exactly: the sums are whole numbers,
so a lost piece, part, row or column shows."""
import pytest

from tests.gpu_util import require_gpu, torch_mod
from tests.int8_rule import few_form, plan
from tests.test_gpu_int8 import guarded, guards_whole

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def wob():
    require_gpu()
    import weight_only_bit_amd as w
    w.device_check()
    return w


# (path, in parts; few rows: waves x groups, weight rows of a workgroup): sizes, ragged in M and N
FORMS = {
    ("few 4 x 1", 8): [(1, 8, 16), (1, 2048, 1024), (5, 2040, 1040), (8, 4088, 4112), (3, 64, 48), (3, 1000, 22800)],
    ("few 8 x 1", 8): [(1, 8392, 5312), (2, 11032, 7696)],
    ("few 2 x 4", 24): [(1, 6000, 2000), (2, 5384, 5392), (7, 6000, 2000), (4, 4104, 16)],
    ("few 2 x 4", 32): [(2, 8192, 1040), (8, 8184, 2000), (5, 6952, 688)],
    ("few 8 x 1 wide", 8): [(16, 1016, 4160), (9, 8, 16), (13, 40, 1232)],
    ("few 8 x 1 wide", 16): [(16, 3000, 2896), (9, 2056, 144), (11, 3464, 256)],
    ("few 4 x 2 wide", 24): [(13, 5760, 2880), (9, 4136, 16), (11, 4768, 464)],
    ("few 4 x 2 wide", 32): [(16, 8184, 1040), (10, 6416, 80), (12, 15392, 240)],
    ("narrow", False): [(17, 8, 16), (40, 2048, 496), (64, 16328, 656)],
    ("narrow", True): [(17, 8, 2016), (17, 72, 1936), (33, 5000, 2896), (100, 2000, 4112), (16, 5376, 21504), (40, 2000, 8192), (33, 1000, 16400)],
    ("small", False): [(71, 9064, 16), (100, 16000, 1040), (129, 8100 // 8 * 8, 2064)],
    ("small", True): [(1094, 264, 7728), (103, 5320, 6768)],
    ("medium", False): [(17, 18136, 16), (200, 16376, 1040), (500, 8184, 2000)],
    ("medium", True): [(100, 5368, 21520), (250, 5376, 8208)],
    # weights that are copied nontemporally
    ("narrow once", False): [(33, 65584, 2064), (61, 11952, 11232)],
    ("narrow once", True): [(17, 6056, 22224)],
    ("small once", False): [(113, 15816, 8512)],
    ("medium once", False): [(100, 27120, 4960)],
    ("medium once", True): [(105, 5728, 23440)],
    ("wide", False): [(133, 18512, 16), (511, 16376, 1040), (1000, 8184, 2064)],
    ("wide", True): [(351, 3024, 20176), (501, 4232, 13504)],
    ("large", False): [(276, 22800, 16), (2047, 16376, 1040), (1500, 5752, 2896)],
    ("large", True): [(140, 16680, 7184), (760, 5376, 21520)],
}
SMALL_SETS = [(form, size) for form, sizes in FORMS.items() for size in sizes]


def named(M, N, K):
    path, parts = plan(M, N, K)
    if path == "few":
        return "few %d x %d%s" % (*few_form(M, N, K), " wide" if M > 8 else ""), parts
    once = M <= {"narrow": 64, "small": 128, "medium": 128}.get(path, 0) and N * K > 128 << 20
    return path + " once" * once, parts > 1


def exact(x, xs, w, ws, bias=None):
    torch = torch_mod()
    y = (x.double() @ w.double().t()).float() * xs[:, None] * ws
    return y if bias is None else y + bias


def inputs(M, N, K, seed):
    torch = torch_mod()
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randint(-128, 128, (M, K), device="cuda", generator=g, dtype=torch.int8)
    w = torch.randint(-128, 128, (N, K), device="cuda", generator=g, dtype=torch.int8)
    return x, torch.rand(M, device="cuda", generator=g) + 0.5, w, torch.rand(N, device="cuda", generator=g) - 0.5


@pytest.mark.parametrize("form,size", SMALL_SETS)
def test_form(wob, form, size):
    torch = torch_mod()
    M, N, K = size
    assert named(M, N, K) == form
    for k in sorted({K, max(16, K - 16), K - K % 128 or K}):
        x, xs, w, ws = inputs(M, N, k, M + N + k)
        buf, out = guarded((M, N), torch.float32, 77)
        need = wob.int8_gemm_workspace_size(M, N, k)
        work = torch.full((max(need, 16) + 64,), 0x7F, dtype=torch.uint8, device="cuda")
        wob.int8_gemm(x, xs, w, ws, out=out, workspace=work[:max(need, 16)])
        want = exact(x, xs, w, ws)
        assert torch.equal(out, want), (k, torch.nonzero(out != want)[:4].tolist())
        assert guards_whole(buf, 77) and bool((work[-64:] == 0x7F).all())
        for dtype in (torch.bfloat16, torch.float16):
            buf, out = guarded((M, N), dtype, 77)
            bias = torch.zeros(N, device="cuda")
            wob.int8_gemm(x, xs, w, ws, bias=bias, out=out, workspace=work[:max(need, 16)])
            assert torch.equal(out, want.to(dtype)) and guards_whole(buf, 77)


@pytest.mark.parametrize("form,size", SMALL_SETS)
def test_bias(wob, form, size):
    """The bias reaches its column; on scales and sums that are powers of two and small whole
    numbers every step is exact."""
    torch = torch_mod()
    M, N, K = size
    x = torch.zeros((M, K), dtype=torch.int8, device="cuda")
    w = torch.zeros((N, K), dtype=torch.int8, device="cuda")
    x[:, -1], w[:, -1] = 2, 3
    x[:, 0] += 1
    w[:, 0] += 1
    xs, ws = torch.full((M,), 0.5, device="cuda"), torch.full((N,), 4.0, device="cuda")
    bias = torch.arange(N, device="cuda").float()
    y = wob.int8_gemm(x, xs, w, ws, bias=bias, out_dtype=torch.float32)
    s = (x[0].double() * w[0].double()).sum().float() * 2.0
    assert torch.equal(y, (s + bias).expand(M, N))
