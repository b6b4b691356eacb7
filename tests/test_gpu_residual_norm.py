"""GPU parity of the norms around a block against block_ref.py, through the binding."""
import numpy as np
import pytest

from tests import block_ref as R
from tests.gpu_util import require_gpu, torch_mod
from tests.test_gpu_int8 import _dt, guarded, guards_whole

pytestmark = pytest.mark.gpu

TYPES = (("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"), ("fp16", "fp32"), ("fp32", "fp32"))


@pytest.fixture(scope="module")
def wob():
    require_gpu()
    import weight_only_bit_amd as w
    w.device_check()
    return w


def inputs(T, H, dtype, res, seed):
    torch = torch_mod()
    g = torch.Generator().manual_seed(seed)
    t = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    dt = _dt(dtype)
    return dict(y=t(T, H).to(dt).cuda(), r=(t(T, H) * 2).to(_dt(res)).cuda(), w=(1 + 0.2 * t(H)).to(dt).cuda(),
                post=(1 + 0.2 * t(H)).to(dt).cuda(), channel=t(H).to(dt).cuda(), rows=t(T, H).to(dt).cuda())


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def want(d, post, gate, alpha, eps, y=True, weight=True):
    return R.norm(f64(d["y"]) if y else None, f64(d["r"]), f64(d["w"]) if weight else None,
                  f64(d["post"]) if post else None, f64(d[gate]) if gate else None,
                  np.float64(np.float32(alpha)), np.float64(np.float32(eps)))


def close(got, ref, bound, dtype):
    off = np.abs(f64(got) - ref)
    ok = off <= bound + R.HALF_STEP[dtype] * (np.abs(ref) + bound) + R.TINY[dtype]
    assert ok.all(), (np.argwhere(~ok)[:5], off[~ok][:5])


@pytest.mark.parametrize("dtype,res", TYPES)
@pytest.mark.parametrize("post", (False, True))
@pytest.mark.parametrize("gate", (None, "channel", "rows"))
@pytest.mark.parametrize("T,H", [(1, 8), (3, 72), (5, 512), (2, 520), (70, 2048), (3, 2056), (300, 5376), (2, 8200),
                                 (2, 32768), (37, 64), (19, 128), (9, 136), (13, 256), (6, 264), (5, 1024), (3, 1032)])
def test_plain(wob, dtype, res, post, gate, T, H):
    torch = torch_mod()
    d = inputs(T, H, dtype, res, T * H)
    h, dh, n, dn = want(d, post, gate, 0.875, 1e-6)
    nb, no = guarded((T, H), _dt(dtype), 77)
    hb, ho = guarded((T, H), _dt(res), 77)
    got = wob.residual_norm(d["y"], d["r"], d["w"], post_weight=d["post"] if post else None,
                            gate=d[gate] if gate else None, alpha=0.875, eps=1e-6, out=no, residual_out=ho)
    torch.cuda.synchronize()
    assert got[0] is no and got[1] is ho and guards_whole(nb, 77) and guards_whole(hb, 77)
    close(ho, h, dh, res)
    close(no, n, dn, dtype)


@pytest.mark.parametrize("dtype,res", TYPES)
@pytest.mark.parametrize("T,H", [(1, 16), (7, 528), (3, 5376), (2, 16384), (2, 32752), (33, 48), (9, 112), (5, 240), (3, 1008)])
def test_int8(wob, dtype, res, T, H):
    torch = torch_mod()
    d = inputs(T, H, dtype, res, T + H)
    h, dh, n, dn = want(d, True, "channel", -1.5, 1e-5)
    cb, c = guarded((T, H), torch.int8, 77)
    sb, s = guarded((T,), torch.float32, 77)
    _, _, ho = wob.residual_norm(d["y"], d["r"], d["w"], post_weight=d["post"], gate=d["channel"], alpha=-1.5,
                                 eps=1e-5, quant=wob.QUANT_INT8, out=c, out_scale=s)
    torch.cuda.synchronize()
    assert guards_whole(cb, 77) and guards_whole(sb, 77)
    close(ho, h, dh, res)
    s64, c64 = f64(s)[:, None], f64(c)
    top, dtop = np.abs(n).max(-1, keepdims=True), dn.max(-1, keepdims=True)
    assert (np.abs(s64 - top / 127) <= dtop / 127 + top / 127 * 2.0 ** -23).all()
    assert (np.abs(c64 * s64 - n) <= (0.5 + 127 * 3 * 2.0 ** -23) * s64 + dn + dtop).all()
    assert (np.abs(c64).max(-1) == 127).all()


@pytest.mark.parametrize("T,H", [(1, 32), (7, 544), (3, 5376), (2, 16384), (40, 2048), (37, 64), (9, 128), (11, 256), (5, 992)])
def test_quantised_rows_are_those_of_the_quantisers(wob, T, H):
    """In 32 bits the normed rows are at hand: the fused codes and scales are byte for byte
    what the quantisers make of them."""
    torch = torch_mod()
    d = inputs(T, H, "fp32", "fp32", H)
    d["r"][0, :8] = 0
    kw = dict(post_weight=d["post"], gate=d["rows"], alpha=0.5)
    n, h = wob.residual_norm(d["y"], d["r"], d["w"], **kw)
    c, s, h8 = wob.residual_norm(d["y"], d["r"], d["w"], quant=wob.QUANT_INT8, **kw)
    qc, qs = wob.int8_quantize(n)
    assert torch.equal(h, h8) and torch.equal(c, qc) and torch.equal(s, qs)
    cb, cv = guarded((T, H // 2), torch.uint8, 77)
    sb, sv = guarded((T, H // 32), torch.uint8, 77)
    c, s, h4 = wob.residual_norm(d["y"], d["r"], d["w"], quant=wob.QUANT_MXFP4, out=cv, out_scale=sv, **kw)
    qc, qs = wob.mxfp4_quantize(n)
    assert torch.equal(h, h4) and torch.equal(c, qc) and torch.equal(s, qs)
    assert guards_whole(cb, 77) and guards_whole(sb, 77)


@pytest.mark.parametrize("dtype,res", TYPES)
def test_mxfp4(wob, dtype, res):
    torch = torch_mod()
    T, H = 9, 2880
    d = inputs(T, H, dtype, res, 4)
    _, _, n, dn = want(d, True, None, 1.0, 1e-6)
    c, s, _ = wob.residual_norm(d["y"], d["r"], d["w"], post_weight=d["post"], quant=wob.QUANT_MXFP4)
    v, scale = R.mxfp4_values(c.cpu().numpy(), s.cpu().numpy())
    block = np.abs(n).reshape(T, -1, 32).max(-1)
    fits = np.repeat((block / 8 * (1 - 1e-5) < scale[:, ::32]) & (scale[:, ::32] <= block / 4 * (1 + 1e-5)), 32, -1)
    assert fits.all()
    # half the distance of neighbouring codes: 1/4 below 2, 1/2 below 4, 1 below 6; 2 above (held at 6)
    a = np.abs(n) / scale
    half = np.where(a < 2, 0.25, np.where(a < 4, 0.5, np.where(a < 6, 1.0, a - 6 + 1e-6)))
    assert (np.abs(v - n) <= half * scale * (1 + 1e-6) + dn).all()


def test_without_a_block(wob):
    torch = torch_mod()
    for dtype, res in TYPES:
        d = inputs(5, 264, dtype, res, 8)
        _, _, n, dn = want(d, False, None, 1.0, 1e-6, y=False)
        got, h = wob.residual_norm(None, d["r"], d["w"])
        assert h is d["r"] and got.dtype == d["w"].dtype
        close(got, n, dn, dtype)


def test_without_a_norm_before(wob):
    torch = torch_mod()
    for dtype, res in TYPES:
        for H in (264, 5376):
            d = inputs(700, H, dtype, res, 8)
            h, dh, _, _ = want(d, True, "rows", 2.0, 1e-6, weight=False)
            n, got = wob.residual_norm(d["y"], d["r"], None, post_weight=d["post"], gate=d["rows"], alpha=2.0)
            assert n is None
            close(got, h, dh, res)


@pytest.mark.parametrize("H", (72, 2048, 5376, 16384))
def test_in_place(wob, H):
    torch = torch_mod()
    d = inputs(33, H, "bf16", "bf16", H)
    n, h = wob.residual_norm(d["y"], d["r"], d["w"], post_weight=d["post"])
    r = d["r"].clone()
    n2, h2 = wob.residual_norm(d["y"], r, d["w"], post_weight=d["post"], residual_out=r)
    assert h2 is r and torch.equal(h, r) and torch.equal(n, n2)


@pytest.mark.parametrize("H", (72, 2048, 5376, 16384))
def test_column_slices(wob, H):
    torch = torch_mod()
    d = inputs(9, 2 * H + 16, "bf16", "fp32", H)
    y, gate = d["y"][:, 8:8 + H], d["y"][:, H + 8:2 * H + 8]
    r, w = d["r"][:, :H].contiguous(), d["w"][:H].contiguous()
    a = wob.residual_norm(y, r, w, gate=gate)
    b = wob.residual_norm(y.contiguous(), r, w, gate=gate.contiguous())
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    with pytest.raises(ValueError):
        wob.residual_norm(d["y"][:, 4:4 + H], r, w)  # rows 8 bytes off
    with pytest.raises(ValueError):
        wob.residual_norm(y, r, w, gate=d["y"][:, 4:4 + H])


@pytest.mark.parametrize("H", (64, 2048, 16384))
def test_special_rows(wob, H):
    """Zeros, infinities and NaN stay in their row; a row of zeros with eps = 0 is NaN, with
    eps > 0 zero."""
    torch = torch_mod()
    d = inputs(6, H, "bf16", "bf16", 2)
    d["y"][0], d["r"][0] = 0, 0
    d["y"][1, 3] = float("nan")
    d["r"][2, H - 1] = float("inf")
    n, h = wob.residual_norm(d["y"], d["r"], d["w"], post_weight=d["post"])
    assert (n[0] == 0).all() and (h[0] == 0).all()
    assert torch.isnan(n[1]).all() and torch.isnan(h[1]).all()
    assert torch.isinf(h[2, H - 1]) and torch.isnan(n[2, H - 1]) and (n[2, :H - 1] == 0).all()
    assert torch.isfinite(n[3:]).all()
    for quant in (wob.QUANT_INT8, wob.QUANT_MXFP4):
        c, s, _ = wob.residual_norm(d["y"], d["r"], d["w"], post_weight=d["post"], quant=quant)
        read = wob.int8_dequant if quant == wob.QUANT_INT8 else wob.mxfp4_dequant
        v = read(c, s)
        assert (v[0] == 0).all() and torch.isnan(v[1]).all() and torch.isnan(v[2, H - 1])
        assert torch.isfinite(v[3:]).all()
    n, _ = wob.residual_norm(d["y"], d["r"], d["w"], eps=0.0)
    assert torch.isnan(n[0]).all()


def test_many_rows(wob):
    """More rows than the grid has workgroups for at once."""
    torch = torch_mod()
    T, H = 4_200_000, 32
    y = torch.randint(-3, 4, (T, H), device="cuda").to(torch.bfloat16)
    r = torch.randint(-3, 4, (T, H), device="cuda").to(torch.bfloat16)
    w = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    n, h = wob.residual_norm(y, r, w)
    assert torch.equal(h, y + r)
    ref = h.float() / torch.sqrt((h.float() ** 2).mean(-1, keepdim=True) + 1e-6)
    assert float((n.float() - ref).abs().max()) <= 6 * 2.0 ** -8
    assert torch.equal(wob.residual_norm(y[-5:], r[-5:], w)[0], n[-5:])


def test_empty(wob):
    torch = torch_mod()
    d = inputs(2, 64, "bf16", "fp32", 2)
    n, h = wob.residual_norm(d["y"][:0], d["r"][:0], d["w"])
    assert n.shape == (0, 64) and h.shape == (0, 64) and h.dtype == torch.float32
    for quant, width in ((wob.QUANT_INT8, 64), (wob.QUANT_MXFP4, 32)):
        c, s, h = wob.residual_norm(d["y"][:0], d["r"][:0], d["w"], post_weight=d["post"], gate=d["rows"][:0], quant=quant)
        assert c.shape == (0, width) and s.shape[0] == 0 and h.shape == (0, 64)
    assert wob.residual_norm(None, d["r"][:0], d["w"])[0].shape == (0, 64)
