"""Refusals of the 8-bit rows and product, the norms around a block and the
group-limited choice: every bad argument is refused before any device access (CPU;
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


def test_int8_quantize_refusals(L):
    def q(x=F.p, dt=1, ldx=64, act=0, c=F.p, s=F.p, R=2, K=64):
        return L.lib().int8_quantize(x, dt, ldx, act, c, s, R, K, None)
    assert q(dt=2) == L.DTYPE and q(dt=7) == L.DTYPE
    for bad in (dict(K=24, ldx=24), dict(K=0), dict(K=-16), dict(K=65552, ldx=65552), dict(R=-1),
                dict(ldx=48), dict(ldx=68), dict(ldx=66, dt=3), dict(act=2), dict(act=1), dict(act=1, ldx=120),
                dict(x=None), dict(c=None), dict(s=None), dict(x=F.odd), dict(c=F.odd), dict(s=F.odd),
                dict(R=1 << 29), dict(ldx=1 << 50)):
        assert q(**bad) == L.INVALID_ARG, bad
    assert q(R=0) == L.OK and q(R=0, x=None, c=None, s=None) == L.OK


def test_int8_dequant_refusals(L):
    def d(c=F.p, s=F.p, o=F.p, dt=1, R=2, K=64):
        return L.lib().int8_dequant(c, s, o, dt, R, K, None)
    assert d(dt=2) == L.DTYPE
    for bad in (dict(K=24), dict(K=0), dict(K=65552), dict(R=-1), dict(R=1 << 29), dict(c=None),
                dict(s=None), dict(o=None), dict(c=F.odd), dict(s=F.odd), dict(o=F.odd)):
        assert d(**bad) == L.INVALID_ARG, bad
    assert d(R=0) == L.OK


def test_int8_gemm_refusals(L):
    def g(x=F.p, xs=F.p, w=F.p, ws=F.p, b=None, y=F.p, dt=1, M=4, N=16, K=64, work=F.p, nb=1 << 40):
        return L.lib().int8_gemm(x, xs, w, ws, b, y, dt, M, N, K, work, nb, None)
    assert g(dt=2) == L.DTYPE
    for bad in (dict(K=24), dict(K=0), dict(K=131072), dict(N=12), dict(M=-1), dict(N=-8), dict(x=None),
                dict(xs=None), dict(w=None), dict(ws=None), dict(y=None), dict(x=F.odd), dict(xs=F.odd),
                dict(w=F.odd), dict(ws=F.odd), dict(b=F.odd), dict(y=F.odd), dict(M=1 << 20, K=1 << 12),
                dict(N=1 << 20, K=1 << 12), dict(M=1 << 40), dict(M=1 << 27, K=16), dict(N=1 << 27, K=16)):
        assert g(**bad) == L.INVALID_ARG, bad
    assert g(M=0) == L.OK and g(N=0) == L.OK
    size = L.lib().int8_gemm_workspace_size
    assert size(-1, 8, 64) == 0 and size(4, -8, 64) == 0 and size(4, 8, 0) == 0 and size(1 << 40, 8, 64) == 0
    assert size(4, 8, 131072) == 0
    for M, N, K in ((1, 16384, 5376), (13, 5760, 2880), (100, 5376, 21504), (16, 512, 65536), (300, 512, 512)):
        need = size(M, N, K)
        if need:
            assert g(M=M, N=N, K=K, nb=need - 1) == L.INVALID_ARG
            assert g(M=M, N=N, K=K, work=None, nb=need) == L.INVALID_ARG
            assert g(M=M, N=N, K=K, work=F.odd, nb=need) == L.INVALID_ARG


def test_residual_norm_refusals(L):
    def r(y=F.p, dt=1, ldy=64, res=F.p, rdt=1, post=None, gate=None, ldg=0, alpha=1.0, w=F.p, eps=1e-6,
          quant=0, n=F.p, ns=None, out=F.p, T=2, H=64):
        return L.lib().residual_norm(y, dt, ldy, res, rdt, post, gate, ldg, alpha, w, eps, quant, n, ns,
                                     out, T, H, None)
    assert r(dt=2) == L.DTYPE and r(rdt=0) == L.DTYPE and r(dt=3, rdt=1) == L.DTYPE and r(rdt=2) == L.DTYPE
    for bad in (dict(H=60), dict(H=0), dict(H=32776, ldy=32776), dict(H=24, quant=1, ns=F.p),
                dict(H=48, quant=2, ns=F.p), dict(T=-1), dict(T=1 << 29), dict(quant=3), dict(quant=1),
                dict(ns=F.p), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
                dict(alpha=float("nan")), dict(alpha=float("inf")), dict(ldy=56), dict(ldy=68),
                dict(gate=F.p, ldg=56), dict(gate=F.p, ldg=68), dict(ldy=1 << 50), dict(gate=F.p, ldg=1 << 50),
                dict(dt=3, rdt=3, ldy=66), dict(y=None, post=F.p), dict(y=None, gate=F.p), dict(y=None, w=None),
                dict(w=None), dict(w=None, n=None, ns=F.p), dict(w=None, n=None, quant=1), dict(res=None),
                dict(out=None), dict(n=None), dict(y=F.odd), dict(res=F.odd), dict(post=F.odd),
                dict(gate=F.odd), dict(w=F.odd), dict(n=F.odd), dict(out=F.odd), dict(quant=1, ns=F.odd)):
        assert r(**bad) == L.INVALID_ARG, bad
    assert r(T=0) == L.OK and r(T=0, w=None, n=None) == L.OK
    # tensors without rows have no address
    assert r(T=0, y=None, post=F.p, gate=F.p, res=None, out=None, n=None, quant=2) == L.OK
    assert r(T=0, H=60) == L.INVALID_ARG and r(T=0, dt=2) == L.DTYPE


def test_moe_route_refusals(L):
    def k(l=F.p, dt=1, b=None, i=F.p, w=F.p, T=2, E=16, topk=2, score=0, groups=4, kept=2, top=2, scale=1.0):
        return L.lib().moe_route(l, dt, b, i, w, T, E, topk, score, groups, kept, top, 1, scale, None)
    assert k(dt=2) == L.DTYPE
    for bad in (dict(T=-1), dict(E=0), dict(E=1025, groups=1, kept=1), dict(E=1028), dict(topk=0), dict(topk=9),
                dict(E=256, topk=65), dict(groups=0), dict(groups=3), dict(groups=128, E=256, kept=64),
                dict(kept=0), dict(kept=5), dict(top=0), dict(top=3), dict(score=2), dict(score=-1),
                dict(scale=float("nan")), dict(scale=float("inf")), dict(T=1 << 25), dict(l=None), dict(i=None),
                dict(w=None), dict(l=F.odd), dict(b=F.odd), dict(i=F.odd), dict(w=F.odd)):
        assert k(**bad) == L.INVALID_ARG, bad
    assert k(T=0) == L.OK


def test_binding_checks(wob):
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="multiple of 16"):
        wob.int8_quantize(x[:, :24].contiguous())
    with pytest.raises(TypeError, match="dtype"):
        wob.int8_quantize(x.double())
    with pytest.raises(ValueError, match="contiguous"):
        wob.int8_quantize(torch.zeros((64, 32), dtype=torch.bfloat16).t()[:, ::2])
    with pytest.raises(ValueError, match="even"):
        wob.int8_quantize(x[:, :63].contiguous(), act=wob.ACT_SILU_MUL)
    with pytest.raises(ValueError, match="activation"):
        wob.int8_quantize(x, act=2)
    with pytest.raises(ValueError, match="device"):
        wob.int8_quantize(x)
    q, s = torch.zeros((4, 64), dtype=torch.int8), torch.zeros(4)
    with pytest.raises(ValueError, match="scale"):
        wob.int8_dequant(q, s[:3])
    with pytest.raises(TypeError, match="codes"):
        wob.int8_dequant(q.to(torch.uint8), s)
    with pytest.raises(TypeError, match="out_dtype"):
        wob.int8_dequant(q, s, out_dtype=torch.int8)
    with pytest.raises(ValueError, match="device"):
        wob.int8_dequant(q, s)
    w, ws = torch.zeros((16, 64), dtype=torch.int8), torch.zeros(16)
    for a, kw, word in (((q, s[:2], w, ws), {}, "x_scale"), ((q, s, w[:, :48], ws), {}, "w_q"),
                        ((q, s, w, ws[:8]), {}, "w_scale"), ((q, s, w, ws), dict(bias=ws[:4]), "bias"),
                        ((q, s, w, ws), dict(out=torch.zeros((4, 8), dtype=torch.bfloat16)), "out"),
                        ((q[0], s, w, ws), {}, "x_q")):
        with pytest.raises(ValueError, match=word):
            wob.int8_gemm(*a, **kw)
    with pytest.raises(TypeError, match="out_dtype"):
        wob.int8_gemm(q, s, w, ws, out_dtype=torch.int32)
    with pytest.raises(TypeError, match="bias"):
        wob.int8_gemm(q, s, w, ws, bias=ws.half())
    with pytest.raises(ValueError, match="device"):
        wob.int8_gemm(q, s, w, ws)


def test_residual_norm_binding_checks(wob):
    y, w = torch.zeros((4, 64), dtype=torch.bfloat16), torch.zeros(64, dtype=torch.bfloat16)
    for a, kw, word in (((y, y[:2], w), {}, "y"), ((y, y, w[:32]), {}, "weight"), ((None, y, None), {}, "nothing"),
                        ((y, y, w), dict(post_weight=w[:8]), "post_weight"), ((y, y, w), dict(gate=w[:8]), "gate"),
                        ((y, y, w), dict(gate=y[:2]), "gate"), ((None, y, w), dict(gate=w), "without y"),
                        ((None, y, w), dict(post_weight=w), "without y"),
                        ((None, y, w), dict(residual_out=y), "without y"),
                        ((y, y, None), dict(quant=1), "without weight"), ((y, y, w), dict(quant=5), "quant"),
                        ((y, y, w), dict(out_scale=w), "out_scale"), ((y.t(), y.t(), w), {}, "contiguous"),
                        ((y[:, :48].contiguous(), y[:, :48].contiguous(), w[:48]), dict(quant=2), "multiple of 32"),
                        ((y, y, w), dict(eps=-1.0), "eps"), ((y, y, w), dict(eps=float("nan")), "eps"),
                        ((y, y, w), dict(alpha=float("inf")), "alpha"),
                        ((y, y, w), dict(out=y[:2]), "out"), ((y, y, w), {}, "device")):
        with pytest.raises(ValueError, match=word):
            wob.residual_norm(*a, **kw)
    with pytest.raises(TypeError, match="residual"):
        wob.residual_norm(y, y.half(), w)
    with pytest.raises(TypeError, match="weight"):
        wob.residual_norm(y, y, w.float())
    with pytest.raises(TypeError, match="dtype"):
        wob.residual_norm(y.double(), y, w)


def test_moe_route_binding_checks(wob):
    l = torch.zeros((4, 16))
    for kw, word in ((dict(topk=0), "topk"), (dict(topk=17), "topk"), (dict(topk=5, groups=4, topk_groups=1), "topk"),
                     (dict(topk=2, groups=3), "groups"), (dict(topk=2, groups=4, topk_groups=5), "topk_groups"),
                     (dict(topk=2, group_top=3), "group_top"), (dict(topk=2, score=7), "score"),
                     (dict(topk=2, bias=torch.zeros(8)), "bias"), (dict(topk=2), "device")):
        with pytest.raises(ValueError, match=word):
            wob.moe_route(l, **kw)
    with pytest.raises(TypeError, match="logits"):
        wob.moe_route(l.int(), 2)
    with pytest.raises(TypeError, match="ids"):
        wob.moe_route(l, 2, ids=torch.zeros((4, 2), dtype=torch.int64))
