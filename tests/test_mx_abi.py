"""Refusals of the MXFP4 quantisation and product, the choice of experts and
the MoE layer: every bad argument is refused before any device access (CPU;
the pointers are host stand-ins)."""
import ctypes
import os

import numpy as np
import pytest
import torch


@pytest.fixture(scope="module")
def L():
    from weight_only_bit_amd import _lib, build
    if not os.path.exists(_lib.LIB_PATH):
        build.build()
    return _lib


@pytest.fixture(scope="module")
def wob(L):
    import weight_only_bit_amd as w
    return w


class _Buf:
    def __init__(self):
        self.buf = np.zeros(128, np.uint8)
        self.p = ctypes.c_void_p(self.buf.ctypes.data + (-self.buf.ctypes.data) % 16)
        self.odd = ctypes.c_void_p(self.p.value + 4)


F = _Buf()


def test_quantize_refusals(L):
    def q(x=F.p, dt=1, ldx=64, c=F.p, s=F.p, R=2, K=64):
        return L.lib().mxfp4_quantize(x, dt, ldx, c, s, R, K, None)
    assert q(dt=2) == L.DTYPE and q(dt=7) == L.DTYPE
    for bad in (dict(K=48), dict(K=0), dict(K=-32), dict(R=-1), dict(ldx=32), dict(ldx=68),
                dict(ldx=66, dt=3), dict(x=None), dict(c=None), dict(s=None), dict(x=F.odd),
                dict(c=F.odd), dict(s=F.odd), dict(R=1 << 30, K=64), dict(ldx=1 << 50),
                dict(K=1 << 40, ldx=1 << 40)):
        assert q(**bad) == L.INVALID_ARG, bad
    assert q(R=0) == L.OK and q(R=0, x=None, c=None, s=None) == L.OK


def test_gemm_refusals(L):
    def g(x=F.p, xs=F.p, w=F.p, ws=F.p, y=F.p, dt=1, M=4, N=16, K=64, work=F.p, nb=1 << 30):
        return L.lib().mxfp4_gemm(x, xs, w, ws, y, dt, M, N, K, work, nb, None)
    assert g(dt=2) == L.DTYPE
    for bad in (dict(K=48), dict(K=0), dict(N=12), dict(M=-1), dict(N=-8), dict(x=None),
                dict(xs=None), dict(w=None), dict(ws=None), dict(y=None), dict(x=F.odd),
                dict(ws=F.odd), dict(y=F.odd), dict(M=1 << 20, K=1 << 14), dict(N=1 << 20, K=1 << 14),
                dict(M=1 << 40)):
        assert g(**bad) == L.INVALID_ARG, bad
    for bad in (dict(M=17, N=(1 << 27) - 16, K=32), dict(M=1 << 26, N=1 << 26, K=32),
                dict(M=1, N=1 << 27, K=32), dict(M=1 << 27, N=8, K=32), dict(M=0, N=1 << 27)):
        assert g(**bad) == L.INVALID_ARG, bad   # M + N below 2^27
    assert g(M=0) == L.OK and g(N=0) == L.OK
    size = L.lib().mxfp4_gemm_workspace_size
    assert size(-1, 8, 64) == 0 and size(4, 8, 0) == 0 and size(1 << 40, 8, 64) == 0
    for M, N, K in ((1, 16384, 5376), (13, 5760, 2880), (100, 5376, 21504), (300, 512, 512)):
        need = size(M, N, K)
        if need:
            assert g(M=M, N=N, K=K, nb=need - 1) == L.INVALID_ARG
            assert g(M=M, N=N, K=K, work=None, nb=need) == L.INVALID_ARG
            assert g(M=M, N=N, K=K, work=F.odd, nb=need) == L.INVALID_ARG


def test_topk_refusals(L):
    def k(l=F.p, dt=1, b=None, i=F.p, w=F.p, T=2, E=8, topk=2):
        return L.lib().moe_topk(l, dt, b, i, w, T, E, topk, 1, None)
    assert k(dt=2) == L.DTYPE
    for bad in (dict(T=-1), dict(E=0), dict(E=4097), dict(topk=0), dict(topk=9), dict(E=128, topk=65),
                dict(T=1 << 40), dict(T=1 << 25, topk=1), dict(l=None), dict(i=None), dict(w=None), dict(l=F.odd),
                dict(b=F.odd), dict(i=F.odd), dict(w=F.odd)):
        assert k(**bad) == L.INVALID_ARG, bad
    assert k(T=0) == L.OK


def test_layer_refusals(L):
    size = L.lib().mxfp4_moe_layer_workspace_size

    def m(x=F.p, l=F.p, dt=1, b=None, w1=F.p, w1s=F.p, w2=F.p, w2s=F.p, y=F.p, T=2, topk=2, E=8,
          H=64, I=64, ws=F.p, nb=1 << 30):
        return L.lib().mxfp4_moe_layer(x, l, dt, b, w1, w1s, w2, w2s, y, T, topk, E, H, I, 1, ws, nb,
                                       None)
    assert m(dt=2) == L.DTYPE
    for bad in (dict(H=96), dict(I=96), dict(H=0), dict(I=0), dict(T=-1), dict(E=0), dict(E=4097),
                dict(topk=9), dict(topk=0), dict(x=None), dict(l=None), dict(w1=None), dict(w1s=None),
                dict(w2=None), dict(w2s=None), dict(y=None), dict(x=F.odd), dict(w1=F.odd),
                dict(w2s=F.odd), dict(y=F.odd), dict(b=F.odd), dict(ws=None), dict(ws=F.odd),
                dict(nb=size(2, 2, 8, 64, 64) - 1), dict(T=1 << 20, H=1 << 12), dict(H=1 << 17, I=1 << 17)):
        assert m(**bad) == L.INVALID_ARG, bad
    assert m(T=0) == L.OK
    assert size(-1, 2, 8, 64, 64) == 0 and size(1, 65, 80, 64, 64) == 0
    assert size(1, 2, 4097, 64, 64) == 0 and size(1, 2, 8, -64, 64) == 0
    assert size(4, 4, 32, 2880, 2880) >= 16 * (4 + 4 + 2 * 2880)


def test_binding_refusals(wob):
    u8, bf, f32 = torch.uint8, torch.bfloat16, torch.float32
    z = torch.zeros
    with pytest.raises(ValueError, match="K=48"):
        wob.mxfp4_quantize(z((2, 48), dtype=bf))
    with pytest.raises(TypeError, match="x has dtype"):
        wob.mxfp4_quantize(z((2, 64), dtype=torch.float64))
    with pytest.raises(ValueError, match="contiguous"):
        wob.mxfp4_quantize(z((64, 64), dtype=bf).t())
    with pytest.raises(ValueError, match="contiguous"):
        wob.mxfp4_quantize(z((1, 64), dtype=bf).expand(4, 64))
    with pytest.raises(ValueError, match="out_scale"):
        wob.mxfp4_quantize(z((2, 64), dtype=bf), out_scale=z((2, 3), dtype=u8))
    with pytest.raises(ValueError, match="device"):
        wob.mxfp4_quantize(z((2, 64), dtype=bf))
    x, xs, w, ws = z((2, 32), dtype=u8), z((2, 2), dtype=u8), z((8, 32), dtype=u8), z((8, 2), dtype=u8)
    with pytest.raises(ValueError, match="x_scale"):
        wob.mxfp4_gemm(x, z((2, 1), dtype=u8), w, ws)
    with pytest.raises(ValueError, match="w_fp4"):
        wob.mxfp4_gemm(x, xs, z((8, 64), dtype=u8), ws)
    with pytest.raises(TypeError, match="out_dtype"):
        wob.mxfp4_gemm(x, xs, w, ws, out_dtype=torch.int32)
    with pytest.raises(TypeError, match="out has dtype"):
        wob.mxfp4_gemm(x, xs, w, ws, out=z((2, 8), dtype=f32), out_dtype=bf)
    with pytest.raises(ValueError, match="device"):
        wob.mxfp4_gemm(x, xs, w, ws)
    with pytest.raises(ValueError, match="topk"):
        wob.moe_topk(z((2, 4)), 5)
    with pytest.raises(TypeError, match="bias"):
        wob.moe_topk(z((2, 4)), 2, bias=z(4, dtype=bf))
    with pytest.raises(TypeError, match="logits"):
        wob.moe_topk(z((2, 4), dtype=torch.int32), 2)
    with pytest.raises(ValueError, match="device"):
        wob.moe_topk(z((2, 4)), 2)
    a = (z((2, 64), dtype=bf), z((2, 4)), 2, z((4, 128, 32), dtype=u8), z((4, 128, 2), dtype=u8),
         z((4, 64, 32), dtype=u8), z((4, 64, 2), dtype=u8))

    def layer(k, v, **kw):
        b = list(a)
        b[k] = v
        return wob.mxfp4_moe_layer(*b, **kw)
    with pytest.raises(ValueError, match="w1_fp4"):
        layer(3, z((4, 64, 32), dtype=u8))
    with pytest.raises(ValueError, match="w2_scale"):
        layer(6, z((4, 64, 3), dtype=u8))
    with pytest.raises(ValueError, match="multiples of 64"):
        layer(0, z((2, 96), dtype=bf))
    with pytest.raises(ValueError, match="x has shape"):
        layer(0, z((3, 64), dtype=bf))
    with pytest.raises(ValueError, match="workspace"):
        layer(0, a[0], workspace=z(4, dtype=u8))
    with pytest.raises(ValueError, match="device"):
        layer(0, a[0])
