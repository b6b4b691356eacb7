"""GPU parity of the group-limited choice of experts against block_ref.py: ids are
equal, weights within their roundings."""
import numpy as np
import pytest

from tests import block_ref as R
from tests.gpu_util import require_gpu, torch_mod
from tests.test_gpu_int8 import _dt, guarded, guards_whole

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def wob():
    require_gpu()
    import weight_only_bit_amd as w
    w.device_check()
    return w


def check(wob, logits, topk, bias=None, sigmoid=True, groups=1, kept=1, top=2, renormalize=True, scale=1.0):
    torch = torch_mod()
    T = logits.shape[0]
    ib, ids = guarded((T, topk), torch.int32, 77)
    wb, weights = guarded((T, topk), torch.float32, 77)
    wob.moe_route(logits, topk, bias=bias, score=wob.SCORE_SIGMOID if sigmoid else wob.SCORE_SOFTMAX, groups=groups,
                  topk_groups=kept, group_top=top, renormalize=renormalize, scale=scale, ids=ids, weights=weights)
    torch.cuda.synchronize()
    assert guards_whole(ib, 77) and guards_whole(wb, 77)
    ref, w = R.route(logits.float().cpu().numpy(), topk, None if bias is None else bias.cpu().numpy(), sigmoid, groups,
                     kept, top, renormalize, np.float64(np.float32(scale)))
    got = ids.cpu().numpy()
    assert np.array_equal(got, ref), (np.argwhere(got != ref)[:5], got[(got != ref).any(-1)][:3])
    off = np.abs(weights.double().cpu().numpy() - w)
    assert (off <= R.route_bound(w, topk)).all(), off.max()
    return got


SIZES = [  # E, groups, kept, topk
    (1, 1, 1, 1), (2, 2, 1, 1), (8, 1, 1, 8), (15, 5, 2, 3), (16, 4, 2, 2), (30, 3, 3, 16), (31, 1, 1, 4), (32, 8, 4, 4),
    (33, 11, 4, 7), (60, 1, 1, 6), (64, 8, 3, 6), (64, 64, 9, 9), (65, 5, 3, 20), (100, 4, 1, 25), (128, 16, 7, 8),
    (160, 8, 3, 6), (192, 3, 2, 64), (200, 25, 8, 8), (256, 8, 4, 8), (256, 1, 1, 32), (257, 1, 1, 8), (384, 12, 5, 10),
    (512, 32, 16, 17), (512, 8, 4, 8), (520, 8, 4, 8), (1000, 50, 20, 16), (1024, 16, 8, 64), (1024, 1, 1, 5), (1023, 33, 31, 8)]


@pytest.mark.parametrize("sigmoid", (True, False))
@pytest.mark.parametrize("E,groups,kept,topk", SIZES)
def test_random(wob, sigmoid, E, groups, kept, topk):
    torch = torch_mod()
    g = torch.Generator().manual_seed(E + topk)
    for T, dtype, biased, top in ((1, "bf16", True, 2), (37, "fp32", True, 2), (70, "fp16", False, 1), (5, "fp32", False, 2)):
        logits = (torch.randn((T, E), generator=g) * 1.5).to(_dt(dtype)).cuda()
        bias = (torch.randn(E, generator=g) * 0.1).cuda() if biased else None
        check(wob, logits, topk, bias, sigmoid, groups, kept, top, renormalize=biased, scale=2.5 if biased else 1.0)


@pytest.mark.parametrize("E,groups,kept,topk", [(16, 4, 2, 3), (60, 6, 2, 5), (256, 8, 4, 8), (512, 8, 4, 12), (1024, 32, 5, 9)])
@pytest.mark.parametrize("sigmoid", (True, False))
def test_masks_and_infinities(wob, E, groups, kept, topk, sigmoid):
    torch = torch_mod()
    g = torch.Generator().manual_seed(E)
    l = torch.randn((12, E), generator=g)
    size = E // groups
    l[0] = -np.inf                       # nothing left
    l[1] = np.nan
    l[2, :] = -np.inf
    l[2, E - 1] = 0.5                    # a single expert
    l[3, :E - size] = -np.inf            # a single group
    l[4, ::2] = -np.inf
    l[5, 3] = np.nan
    l[6, 1] = np.inf
    l[7, :size] = np.inf
    l[8] = -3.0e38                       # finite, but scores of zero
    l[9] = torch.finfo(torch.float32).min
    l[9, 2] = 0
    l[10, : E // 2] = -120.0
    l[11] = 40.0                         # sigmoid: equal scores of one
    bias = torch.randn(E, generator=g) * 0.1
    for b in (None, bias):
        for renormalize in (True, False):
            ids = check(wob, l.cuda(), topk, None if b is None else b.cuda(), sigmoid, groups, kept, 2, renormalize)
            assert (ids[:2] == -1).all() and ids[2, 0] == E - 1 and (ids[2, 1:] == -1).all()
    bias[1], bias[2], bias[5] = -np.inf, np.nan, np.inf
    check(wob, l[3:].cuda(), topk, bias.cuda(), sigmoid, groups, kept, 2)
    check(wob, l[3:].cuda(), topk, bias.cuda(), sigmoid, groups, kept, 1)


@pytest.mark.parametrize("E,groups,kept,topk", [(15, 3, 2, 6), (64, 8, 4, 8), (256, 8, 4, 8), (256, 16, 3, 40), (1024, 8, 2, 64)])
def test_ties(wob, E, groups, kept, topk):
    """Equal scores and equal group sums go to the lowest index."""
    torch = torch_mod()
    g = torch.Generator().manual_seed(E)
    l = torch.randint(-1, 2, (40, E), generator=g).float()
    l[0] = 0
    l[1, ::2] = -0.0
    b = torch.randint(0, 2, (E,), generator=g).float()
    for bias in (None, b.cuda()):
        for top in (1, 2):
            for sigmoid in (True, False):
                check(wob, l.cuda(), topk, bias, sigmoid, groups, kept, top)


def test_values_next_to_a_border(wob):
    """Scores that differ in the last places: the order is that of correctly rounded ones."""
    torch = torch_mod()
    g = torch.Generator().manual_seed(5)
    T, E = 600, 256
    l = (0.7 + torch.randint(-40, 41, (T, E), generator=g) * 2.0 ** -23).float()
    b = torch.randint(0, 8, (E,), generator=g) * 2.0 ** -24
    check(wob, l.cuda(), 8, b.float().cuda(), True, 8, 4, 2)
    check(wob, l.cuda(), 8, b.float().cuda() * 2.0 ** -8, False, 8, 4, 2)


@pytest.mark.parametrize("sigmoid", (True, False))
@pytest.mark.parametrize("E,groups,kept,topk", SIZES)
def test_many_rows_of_every_kind(wob, sigmoid, E, groups, kept, topk):
    """Past 2048 tokens up to 16 lanes share a token: random, tied, masked and infinite rows,
    many times over, so that every row meets every place of a wave."""
    torch = torch_mod()
    g = torch.Generator().manual_seed(3 * E + topk)
    base = torch.randn((41, E), generator=g) * 1.5
    base[5:15] = torch.randint(-1, 2, (10, E), generator=g).float()
    base[15] = 0
    base[16] = -np.inf
    base[17, ::2] = -np.inf
    base[18, : E - 1] = np.nan
    base[19, E // 2:] = np.inf
    base[20] = 50.0
    base[21] = -300.0
    base[22:26] = (0.7 + torch.randint(-9, 10, (4, E), generator=g) * 2.0 ** -23)
    reps = 53
    for dtype, biased, top, renormalize in (("fp32", True, 2, True), ("bf16", False, 1, False), ("fp16", True, 1, True)):
        logits = base.to(_dt(dtype)).cuda()
        bias = (torch.randint(-4, 5, (E,), generator=g).float() * 0.0625) if biased else None
        ids, w = R.route(logits.float().cpu().numpy(), topk, None if bias is None else bias.numpy(), sigmoid, groups, kept,
                         top, renormalize, 1.0)
        bias = None if bias is None else bias.cuda()
        got = wob.moe_route(logits.repeat(reps, 1), topk, bias=bias,
                            score=wob.SCORE_SIGMOID if sigmoid else wob.SCORE_SOFTMAX, groups=groups, topk_groups=kept,
                            group_top=top, renormalize=renormalize)
        assert reps * 41 > 2048
        i = got[0].view(reps, 41, topk).cpu().numpy()
        assert (i == ids).all(), (dtype, np.argwhere((i != ids).any(-1))[:4])
        off = np.abs(got[1].view(reps, 41, topk).double().cpu().numpy() - w)
        assert (off <= R.route_bound(w, topk)).all()


def test_one_group_and_kept_all_are_the_same(wob):
    torch = torch_mod()
    l = torch.randn((300, 96), device="cuda")
    a = wob.moe_route(l, 6)
    b = wob.moe_route(l, 6, groups=8, topk_groups=8)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_softmax_without_groups_is_the_choice_of_experts(wob):
    """moe_topk with its bias of None chooses the same experts (its order is that of the
    logits; here all scores differ in binary32)."""
    torch = torch_mod()
    l = torch.stack([torch.randperm(64) for _ in range(200)]).float().cuda() * 0.1
    for renormalize in (True, False):
        a = wob.moe_route(l, 8, score=wob.SCORE_SOFTMAX, renormalize=renormalize)
        b = wob.moe_topk(l, 8, renormalize=renormalize)
        assert torch.equal(a[0], b[0]) and float((a[1] / b[1] - 1).abs().max()) <= 2.0 ** -18


def test_many_tokens(wob):
    torch = torch_mod()
    g = torch.Generator().manual_seed(1)
    l = torch.randn((3001, 64), generator=g)
    check(wob, l.cuda(), 6, (torch.randn(64, generator=g) * 0.1).cuda(), True, 8, 4, 2)
    big = l.cuda().repeat(40, 1)
    ids, w = wob.moe_route(big, 6, groups=8, topk_groups=4)
    one, v = wob.moe_route(l.cuda(), 6, groups=8, topk_groups=4)
    assert torch.equal(ids, one.repeat(40, 1)) and torch.equal(w, v.repeat(40, 1))


def test_empty(wob):
    torch = torch_mod()
    ids, w = wob.moe_route(torch.zeros((0, 16), device="cuda"), 2)
    assert ids.shape == (0, 2) and w.shape == (0, 2)
