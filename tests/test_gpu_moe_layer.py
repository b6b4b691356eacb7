"""GPU parity of the choice of experts and the mixture-of-experts layer against
the 64-bit references of mx_ref.py, through the binding."""
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


def _dt(name):
    torch = torch_mod()
    return {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[name]


def _choice(wob, logits, topk, bias=None, renormalize=True):
    """Checked wob.moe_topk of a host tensor; the device outputs."""
    torch = torch_mod()
    T = logits.shape[0]
    ids = torch.full((T + 8, topk), 77, dtype=torch.int32, device="cuda")
    w = torch.full((T + 8, topk), float("nan"), dtype=torch.float32, device="cuda")
    lo = 4  # four guard rows in front keep 16-byte alignment
    wob.moe_topk(logits.cuda(), topk, bias=None if bias is None else bias.cuda(),
                 renormalize=renormalize, ids=ids[lo:lo + T], weights=w[lo:lo + T])
    torch.cuda.synchronize()
    assert (ids[:lo] == 77).all() and (ids[lo + T:] == 77).all()
    assert torch.isnan(w[:lo]).all() and torch.isnan(w[lo + T:]).all()
    ids, w = ids[lo:lo + T].cpu().numpy(), w[lo:lo + T].cpu().numpy()
    rid, rw, spread = R.choose(logits.float().numpy(), topk, None if bias is None else bias.numpy(),
                               renormalize)
    assert np.array_equal(ids, rid), np.argwhere(ids != rid)[:4]
    off = np.abs(w - rw)
    assert (off <= R.choice_bound(rw, spread, logits.shape[1])).all(), float(off.max())


@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("T,E,topk,dtype", [(1, 1, 1, "fp32"), (1, 32, 4, "bf16"), (3, 5, 5, "fp16"),
                                            (65, 8, 2, "bf16"), (130, 63, 8, "fp32"), (67, 64, 1, "fp32"),
                                            (41, 65, 16, "bf16"), (77, 128, 6, "fp16"),
                                            (50, 256, 8, "fp32"), (9, 300, 64, "bf16"),
                                            (21, 513, 7, "fp32"), (5, 1024, 64, "fp16"),
                                            (3, 4096, 10, "fp32"), (300, 16, 16, "bf16"),
                                            (1000, 4, 2, "fp32")])
def test_choice_random(wob, T, E, topk, dtype, renormalize):
    torch = torch_mod()
    g = torch.Generator().manual_seed(T * E + topk)
    l = (torch.randn((T, E), generator=g) * 2).to(_dt(dtype))
    _choice(wob, l, topk, None, renormalize)
    _choice(wob, l, topk, torch.randn(E, generator=g), renormalize)


@pytest.mark.parametrize("E,topk", [(6, 4), (32, 4), (100, 16), (256, 8), (700, 9)])
def test_choice_ties_go_to_the_lowest_expert(wob, E, topk):
    torch = torch_mod()
    g = torch.Generator().manual_seed(E)
    l = torch.randint(-2, 3, (60, E), generator=g).float()   # many equal scores
    l[torch.rand((60, E), generator=g) < 0.2] = -0.0          # zeros of both signs are equal
    _choice(wob, l, topk)
    _choice(wob, torch.zeros((3, E)), topk, None, False)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("E,topk", [(5, 3), (32, 4), (64, 8), (200, 12)])
def test_choice_masks(wob, dtype, E, topk):
    """Masked experts, rows with fewer than topk left, rows with none, NaN, infinities and the
    type's lowest value as a mask."""
    torch = torch_mod()
    g = torch.Generator().manual_seed(E + topk)
    l = (torch.randn((40, E), generator=g) * 3).to(_dt(dtype))
    inf = float("inf")
    l[:20][torch.rand((20, E), generator=g) < 0.6] = -inf
    l[1] = -inf
    l[2] = -inf
    l[2, E - 1] = 0.5
    l[3] = float("nan")
    l[4, ::2] = float("nan")
    l[5, 1] = inf
    l[6, 1], l[6, 3] = inf, inf
    l[7] = torch.finfo(_dt(dtype)).min
    l[8] = torch.finfo(_dt(dtype)).min
    l[8, 2] = 1.0
    l[9] = inf
    for renormalize in (True, False):
        _choice(wob, l, topk, None, renormalize)
    bias = torch.randn(E, generator=g)
    bias[0], bias[E - 1] = -inf, float("nan")
    _choice(wob, l, topk, bias)
    _choice(wob, l, topk, torch.full((E,), -inf))


@pytest.mark.parametrize("E,topk", [(3, 2), (32, 4), (33, 8), (128, 3), (256, 8), (260, 8)])
def test_choice_zeros_of_both_signs_are_equal_scores(wob, E, topk):
    """-0 + -0 is -0 and 0 + -0 is 0: the same score, so the lowest expert comes first."""
    torch = torch_mod()
    g = torch.Generator().manual_seed(E)
    l = torch.where(torch.rand((50, E), generator=g) < 0.5, 0.0, -0.0)
    _choice(wob, l, topk, torch.full((E,), -0.0))
    _choice(wob, l, topk, torch.zeros(E), False)
    _choice(wob, l, topk)


@pytest.mark.parametrize("E", [64, 100, 128, 200, 256, 512])
@pytest.mark.parametrize("topk", [8, 16, 17])
def test_choice_ties_in_some_rows(wob, E, topk):
    """Rows with equal scores at, above and below the last place, beside rows without."""
    torch = torch_mod()
    g = torch.Generator().manual_seed(E + topk)
    l = torch.randn((96, E), generator=g)
    top = l.sort(-1, descending=True).values
    l[3, 0] = l[3, E - 1] = top[3, topk - 1]      # a second one at the last place
    l[9, 5], l[9, 50] = top[9, 0] + 1, top[9, 0] + 1
    l[17, 7] = l[17, 8] = top[17, -1] - 1          # far below it
    l[33] = 0.25
    l[34, :-3] = -float("inf")
    _choice(wob, l, topk)
    _choice(wob, l, topk, None, False)


def test_choice_empty_batch(wob):
    torch = torch_mod()
    ids, w = wob.moe_topk(torch.empty((0, 8), device="cuda"), 2)
    assert ids.shape == (0, 2) and w.shape == (0, 2)


# ---- the layer ---------------------------------------------------------------

def _layer_inputs(T, E, H, I, seed, lo=117, hi=121):
    rng = np.random.default_rng(seed)
    torch = torch_mod()
    x = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).to(torch.bfloat16)
    logits = torch.from_numpy((rng.standard_normal((T, E)) * 1.5).astype(np.float32))
    w = (rng.integers(0, 256, (E, 2 * I, H // 2), np.uint8), rng.integers(lo, hi + 1, (E, 2 * I, H // 32), np.uint8),
         rng.integers(0, 256, (E, H, I // 2), np.uint8), rng.integers(lo, hi + 1, (E, H, I // 32), np.uint8))
    return x, logits, w


def _layer(wob, x, logits, topk, w, bias=None, renormalize=True, wd=None):
    torch = torch_mod()
    T, H = x.shape
    out = torch.full((T + 2, H), float("nan"), dtype=torch.bfloat16, device="cuda")
    wd = wd or [dev(a) for a in w]
    need = wob.moe_layer_workspace_size(T, topk, logits.shape[1], H, w[2].shape[2] * 2)
    work = torch.full((need + 32,), 0xFF, dtype=torch.uint8, device="cuda")
    wob.mxfp4_moe_layer(x.cuda(), logits.cuda(), topk, *wd, bias=None if bias is None else bias.cuda(),
                        renormalize=renormalize, out=out[1:T + 1], workspace=work[:need])
    torch.cuda.synchronize()
    assert torch.isnan(out[0]).all() and torch.isnan(out[-1]).all(), "write outside y"
    assert (work[need:] == 0xFF).all(), "write past the workspace"
    return out[1:-1].double().cpu().numpy()


def _check_layer(wob, x, logits, topk, w, bias=None, renormalize=True):
    y = _layer(wob, x, logits, topk, w, bias, renormalize)
    ids, p, _ = R.choose(logits.float().numpy(), topk, None if bias is None else bias.numpy(), renormalize)
    ref, bound = R.layer(x.double().numpy(), ids, p, *w)
    off, tol = np.abs(y - ref), R.rounded(ref, bound, "bf16")
    assert (off <= tol).all(), (np.argwhere(~(off <= tol))[:4], float((off / tol).max()))


@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 7, 8, 9, 12, 16, 17, 20, 31, 32, 33, 40, 70])
@pytest.mark.parametrize("E,topk,H,I", [(4, 2, 128, 64), (8, 3, 192, 320), (32, 4, 576, 448)])
def test_layer_random(wob, T, E, topk, H, I):
    x, logits, w = _layer_inputs(T, E, H, I, T + E)
    _check_layer(wob, x, logits, topk, w)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T", [1, 6, 24])
@pytest.mark.parametrize("renormalize", [True, False])
def test_layer_logit_types_and_bias(wob, dtype, T, renormalize):
    torch = torch_mod()
    x, logits, w = _layer_inputs(T, 16, 256, 192, 11)
    bias = torch.randn(16, generator=torch.Generator().manual_seed(3))
    _check_layer(wob, x, logits.to(_dt(dtype)), 4, w, bias, renormalize)


@pytest.mark.parametrize("T,E,topk", [(1, 1, 1), (8, 1, 1), (32, 1, 1), (33, 2, 2), (4, 64, 64), (2, 100, 8),
                                      (40, 3, 1), (16, 300, 16)])
def test_layer_few_and_many_experts(wob, T, E, topk):
    x, logits, w = _layer_inputs(T, E, 128, 64, T * E)
    _check_layer(wob, x, logits, topk, w)


@pytest.mark.parametrize("T", [1, 5, 32, 48])
def test_layer_every_token_on_the_same_experts(wob, T):
    """All rows meet in the same experts: the fullest expert holds T rows."""
    x, logits, w = _layer_inputs(T, 8, 192, 128, T)
    logits[:, 3] += 50
    logits[:, 5] += 40
    _check_layer(wob, x, logits, 2, w)


@pytest.mark.parametrize("T", [1, 4, 20, 40])
def test_layer_masked_rows(wob, T):
    """A token whose scores are all masked gets a zero row; one with fewer than topk experts
    left sums those; a NaN score is no expert."""
    inf = float("inf")
    x, logits, w = _layer_inputs(T, 8, 128, 128, 5)
    logits[0] = -inf
    if T > 2:
        logits[1] = -inf
        logits[1, 6] = 0.1
        logits[2, ::2] = float("nan")
    _check_layer(wob, x, logits, 3, w)
    assert (_layer(wob, x, logits, 3, w)[0] == 0).all()


@pytest.mark.parametrize("T", [1, 3, 32])
def test_layer_unchosen_experts_are_not_read_into_the_result(wob, T):
    """NaN scales in experts that no token chose reach no output, and a chosen one's reach
    only the tokens that chose it."""
    x, logits, w = _layer_inputs(T, 6, 128, 64, 21)
    logits[:, 4] = -float("inf")
    logits[:, 2] = -float("inf")
    logits[0, 2] = 30.0
    w[1][4], w[3][4] = 255, 255
    ids, _, _ = R.choose(logits.numpy(), 2)
    assert np.isfinite(_layer(wob, x, logits, 2, w)).all()
    w[3][2] = 255
    y = _layer(wob, x, logits, 2, w)
    hit = (ids == 2).any(1)
    assert np.isnan(y[hit]).all() and np.isfinite(y[~hit]).all()


@pytest.mark.parametrize("T", [1, 8, 24, 40])
def test_layer_a_nan_token_stays_alone(wob, T):
    x, logits, w = _layer_inputs(T, 4, 128, 64, 2)
    x[T - 1, 5] = float("nan")
    y = _layer(wob, x, logits, 2, w)
    assert np.isnan(y[T - 1]).all() and np.isfinite(y[:T - 1]).all()


def test_layer_empty_batch(wob):
    torch = torch_mod()
    x, logits, w = _layer_inputs(1, 4, 64, 64, 2)
    y = wob.mxfp4_moe_layer(x[:0].cuda(), logits[:0].cuda(), 2, *(dev(a) for a in w))
    assert y.shape == (0, 64)


@pytest.mark.parametrize("T", [1, 4, 32])
def test_layer_full_size(wob, T):
    """32 experts, top-4, H = I = 2880: every output."""
    x, logits, w = _layer_inputs(T, 32, 2880, 2880, T)
    _check_layer(wob, x, logits, 4, w)


@pytest.mark.parametrize("T", [1, 6, 32, 40])
def test_layer_is_the_three_calls(wob, T):
    """Within the bound of the layer's own sums the same as choice, stage 1 and stage 2 in turn."""
    torch = torch_mod()
    x, logits, w = _layer_inputs(T, 8, 256, 192, 8)
    wd = [dev(a) for a in w]
    ids, p = wob.moe_topk(logits.cuda(), 3)
    a = wob.mxfp4_moe_gemm(x.cuda(), ids, wd[0], wd[1], act=wob.ACT_SILU_MUL)
    y = wob.mxfp4_moe_stage2(a, ids, p, wd[2], wd[3]).double().cpu().numpy()
    rid, rp, _ = R.choose(logits.numpy(), 3)
    ref, bound = R.layer(x.double().numpy(), rid, rp, *w)
    tol = R.rounded(ref, bound, "bf16")
    assert (np.abs(y - ref) <= tol).all()
    assert (np.abs(_layer(wob, x, logits, 3, w, wd=wd) - y) <= 2 * tol).all()


@pytest.mark.parametrize("T", [1, 7, 24, 40])
def test_layer_captured_and_replayed(wob, T):
    """The whole path as it is used: weights quantised, then the layer captured in a graph and
    replayed over changing inputs; every replay equals the eager result bit for bit, with a
    dirty workspace and on another stream."""
    torch = torch_mod()
    E, H, I, topk = 8, 320, 256, 3
    g = torch.Generator().manual_seed(T)
    w1, w1s = wob.mxfp4_quantize((torch.randn((E, 2 * I, H), generator=g) * 0.1).to(torch.bfloat16).cuda())
    w2, w2s = wob.mxfp4_quantize((torch.randn((E, H, I), generator=g) * 0.1).to(torch.bfloat16).cuda())
    x = torch.randn((T, H), generator=g).to(torch.bfloat16).cuda()
    logits = torch.randn((T, E), generator=g).to(torch.bfloat16).cuda()
    work = torch.empty(wob.moe_layer_workspace_size(T, topk, E, H, I), dtype=torch.uint8, device="cuda")
    y = wob.mxfp4_moe_layer(x, logits, topk, w1, w1s, w2, w2s, workspace=work)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        wob.mxfp4_moe_layer(x, logits, topk, w1, w1s, w2, w2s, out=y, workspace=work)
    side = torch.cuda.Stream()
    for k in range(4):
        x.copy_(torch.randn((T, H), generator=g).to(torch.bfloat16).cuda())
        logits.copy_(torch.randn((T, E), generator=g).to(torch.bfloat16).cuda())
        y.fill_(float("nan"))
        work.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            want = wob.mxfp4_moe_layer(x, logits, topk, w1, w1s, w2, w2s)
        side.synchronize()
        assert torch.equal(y, want), k
    ref_in = [t.cpu().numpy() for t in (w1, w1s, w2, w2s)]
    ids, p, _ = R.choose(logits.float().cpu().numpy(), topk)
    ref, bound = R.layer(x.double().cpu().numpy(), ids, p, *ref_in)
    off = np.abs(y.double().cpu().numpy() - ref)
    assert (off <= R.rounded(ref, bound, "bf16")).all()


@pytest.mark.parametrize("T,E,topk,H,I", [
    (64, 16, 8, 128, 64), (65, 16, 8, 128, 64), (64, 16, 9, 128, 64),    # tokens, pairs at their limits
    (8, 70, 64, 64, 64), (9, 70, 64, 64, 64), (57, 33, 9, 192, 64),
    (5, 256, 6, 64, 128), (5, 257, 6, 64, 128), (1, 256, 64, 64, 64),    # experts
    (1, 3, 2, 4160, 64), (3, 3, 2, 8192, 64), (9, 2, 1, 6208, 192),      # rows of several rounds
    (1, 3, 2, 64, 4160), (3, 3, 2, 64, 8192), (9, 2, 1, 192, 6208),
    (8, 2, 2, 8512, 64), (8, 2, 2, 8576, 64), (8, 2, 2, 64, 8576),       # the staged rows' limit
    (1, 4, 4, 64, 4096), (1, 70, 34, 128, 1792), (1, 70, 35, 128, 1792), (1, 2, 2, 64, 32768),
    (4, 9, 3, 128, 2112), (5, 9, 3, 128, 2112), (8, 9, 3, 128, 2048), (9, 9, 3, 128, 2048),
    (4, 40, 34, 128, 1792), (4, 40, 35, 128, 1792), (3, 5, 2, 2048, 2112), (12, 5, 2, 1024, 1088),
    (1, 2, 2, 32768, 64), (1, 2, 2, 32832, 64), (1, 2, 1, 64, 32768), (1, 2, 1, 64, 32832)])
def test_layer_at_the_limits_of_its_kernels(wob, T, E, topk, H, I):
    """On both sides of every limit of the kernels for few tokens."""
    x, logits, w = _layer_inputs(T, E, H, I, T + E + topk)
    _check_layer(wob, x, logits, topk, w)


@pytest.mark.parametrize("T", [1, 3, 8])
@pytest.mark.parametrize("left", [0, 1, 2, 4, 5])
@pytest.mark.parametrize("E,H,I", [(9, 128, 64), (40, 64, 1408)])
def test_layer_with_experts_left(wob, T, E, H, I, left):
    """Tokens for which fewer experts than places are left, down to none."""
    x, logits, w = _layer_inputs(T, E, H, I, left)
    logits[:, left:] = -float("inf")
    logits[T // 2:, 3] = -float("inf")
    for renormalize in (True, False):
        _check_layer(wob, x, logits, 5, w, None, renormalize)


@pytest.mark.parametrize("T", [1, 12])
def test_layer_on_two_streams_at_once(wob, T):
    """Calls without a common workspace do not disturb each other."""
    torch = torch_mod()
    E, topk, H, I = 16, 4, 1024, 768
    sets = []
    for seed in (1, 2):
        x, logits, w = _layer_inputs(T, E, H, I, seed)
        sets.append((x.cuda(), logits.cuda(), topk, *(dev(a) for a in w)))
    want = [wob.mxfp4_moe_layer(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[], []]
    for _ in range(20):
        for i, (st, s) in enumerate(zip(streams, sets)):
            with torch.cuda.stream(st):
                got[i].append(wob.mxfp4_moe_layer(*s))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(want[i], y) for y in got[i])


@pytest.mark.parametrize("T", [1, 20, 70])
def test_layer_captured_with_its_own_workspace(wob, T):
    """Captured without a workspace of the caller's: the graph's memory pool holds it."""
    torch = torch_mod()
    E, topk, H, I = 8, 2, 256, 128
    x, logits, w = _layer_inputs(T, E, H, I, 77)
    x, logits, wd = x.cuda(), logits.cuda(), [dev(a) for a in w]
    want = wob.mxfp4_moe_layer(x, logits, topk, *wd)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = wob.mxfp4_moe_layer(x, logits, topk, *wd)
    for _ in range(3):
        y.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
        assert torch.equal(wob.mxfp4_moe_layer(x, logits, topk, *wd), want)


def test_choice_offsets_past_32_bits(wob):
    """More than 2^31 scores: the last rows, and one in the middle."""
    torch = torch_mod()
    T, E, topk = 530000, 4096, 3
    l = torch.zeros((T, E), dtype=torch.bfloat16, device="cuda")
    rows = torch.tensor([0, 1, T // 2, 524288, 524289, T - 1], device="cuda")
    l[rows, torch.tensor([5, 4095, 17, 3, 2048, 4094], device="cuda")] = 2.0
    l[rows, torch.tensor([6, 0, 4000, 4, 1, 9], device="cuda")] = 1.0
    ids, w = wob.moe_topk(l, topk)
    got, rest = ids[rows].cpu().tolist(), ids[1000].cpu().tolist()
    assert got == [[5, 6, 0], [4095, 0, 1], [17, 4000, 0], [3, 4, 0], [2048, 1, 0], [4094, 9, 0]]
    assert rest == [0, 1, 2]
    # exp of -1 and -2 to 2^-21 (argument, exponential), sum and quotient to 2^-22
    want = torch.softmax(torch.tensor([2.0, 1.0, 0.0], dtype=torch.float64), 0)
    assert (w[rows].cpu().double() - want).abs().max() <= 2.0 ** -20


def test_choice_on_two_streams_at_once(wob):
    torch = torch_mod()
    g = torch.Generator().manual_seed(4)
    ls = [torch.randn((4000, 128), generator=g).cuda() for _ in range(2)]
    want = [wob.moe_topk(l, 8) for l in ls]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in ls], [[], []]
    for _ in range(10):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(wob.moe_topk(ls[i], 8))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, want[i][0]) and torch.equal(b, want[i][1]) for a, b in got[i])
