"""MI355X (gfx950) weight-only 4-bit GEMM: Python binding of the C-ABI library.

Argument marshalling only: tensors supply device memory and
``torch.cuda.current_stream()`` supplies the stream; every step of the
computation runs in the library's HIP kernels (``csrc/``).  There is no CPU
fallback.

    y = gemm(x, qweight, scales, qzeros, group_size)        # W4A16
    y = gemm_grouped(x, m_offsets, qweight, scales, qzeros, group_size)
    y = mxfp4_moe_gemm(x, topk_ids, w_fp4, w_scale)         # MoE stage 1
    y = mxfp4_moe_stage2(a, topk_ids, topk_weights, w2_fp4, w2_scale)  # MoE stage 2
    ids, weights = moe_topk(logits, topk)                   # the choice of experts
    y = mxfp4_moe_layer(x, logits, topk, w1_fp4, w1_scale, w2_fp4, w2_scale)  # a whole MoE layer
    codes, scale = mxfp4_quantize(x)                        # 16/32-bit rows -> MXFP4
    y = mxfp4_gemm(x_fp4, x_scale, w_fp4, w_scale)          # MXFP4 x MXFP4
    codes, scale = int8_quantize(x)                         # 16/32-bit rows -> int8 rows
    y = int8_gemm(x_q, x_scale, w_q, w_scale)               # int8 x int8, scales per row and column
    n, h = residual_norm(y, residual, weight)               # the norms around a block
    ids, weights = moe_route(logits, topk, bias, groups=8, topk_groups=4)  # group-limited choice

Layouts are those of ``include/weight_only_bit.h``.
"""
from __future__ import annotations

import functools
import math

from . import _lib
from ._lib import (ACT_NONE, ACT_SILU_MUL, BF16, DTYPE, F16, F32, INVALID_ARG, OK, PATH_AUTO,
                   PATH_SKINNY, PATH_TILED, QUANT_INT8, QUANT_MXFP4, QUANT_NONE, SCORE_SIGMOID,
                   SCORE_SOFTMAX, U4X8_I32, UNSUPPORTED, WobArgError, WobDtypeError, WobError)

__all__ = [
    "gemm", "gemm_grouped", "mxfp4_moe_gemm", "moe_workspace_size", "mxfp4_moe_stage2",
    "moe_stage2_workspace_size", "moe_topk", "mxfp4_moe_layer", "moe_layer_workspace_size",
    "mxfp4_quantize", "mxfp4_gemm", "mxfp4_gemm_workspace_size", "int8_quantize",
    "int8_dequant", "int8_gemm", "int8_gemm_workspace_size", "residual_norm", "moe_route",
    "w4a16_dequant", "mxfp4_dequant", "stream_read", "device_check", "WobError", "WobDtypeError",
    "WobArgError", "PATH_AUTO", "PATH_SKINNY", "PATH_TILED", "ACT_NONE", "ACT_SILU_MUL",
    "QUANT_NONE", "QUANT_INT8", "QUANT_MXFP4", "SCORE_SIGMOID", "SCORE_SOFTMAX",
]


_torch_mod = None
_tags = None
_raw_stream = _get_device = _empty_here = _values = _bytes = _int8 = _fp32 = None
_value_tags = None
_loaded = None  # the library, once an operator has been called


def _torch():
    """torch, imported on first use; the dtype tags and the device and stream queries with it."""
    global _torch_mod, _tags, _values, _bytes, _int8, _fp32, _raw_stream, _get_device, _empty_here
    global _value_tags
    if _torch_mod is None:
        import torch
        _tags = {torch.float16: F16, torch.bfloat16: BF16, torch.int32: U4X8_I32,
                 torch.float32: F32}
        _values, _bytes = (torch.float16, torch.bfloat16, torch.float32), (torch.uint8,)
        _int8, _fp32 = (torch.int8,), (torch.float32,)
        _value_tags = {t: _tags[t] for t in _values}
        # the current stream's handle without building a Stream object: 0.1
        # against 1.9 us, in calls whose launch takes 3
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda index: torch.cuda.current_stream(index).cuda_stream)
        _get_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
        # a tensor (shape, strides, dtype) on the current device: 0.8 against 1.7 us
        guards = getattr(getattr(torch._C, "_dynamo", None), "guards", None)
        _empty_here = getattr(guards, "_empty_strided_cuda", None) or (
            lambda shape, strides, dtype: torch.empty_strided(shape, strides, dtype=dtype, device="cuda"))
        _torch_mod = torch
    return _torch_mod


def _tag(t):
    _torch()
    return _tags.get(t.dtype, -1)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _run(fn, device, *args):
    """fn(*args, stream) with `device` current, on its current stream.  (Entering
    torch.cuda.device costs 1.3 us, so it is done only where it changes the device.)"""
    index = device.index
    if _get_device() == index:
        return fn(*args, _raw_stream(index))
    with _torch_mod.cuda.device(index):
        return fn(*args, _raw_stream(index))


def _check_device(*tensors):
    first, index = None, -1
    for t in tensors:
        if t is None:
            continue
        at = t.get_device()
        if at < 0:  # a host tensor
            raise ValueError("all operands must be device tensors")
        if not t.is_contiguous():
            raise ValueError("all operands must be contiguous")
        if first is None:
            first, index = t, at
        elif at != index:
            raise ValueError("operands live on different devices")
    return None if first is None else first.device


# Shape and dtype checks.  They read only .shape and .dtype, so they run
# before any device access (and work on CPU or meta tensors): the C ABI sees
# raw pointers and could not detect an operand smaller than its shape says.

def _want(t, name, shape, dtypes):
    """t must exist, have exactly `shape`, and one of `dtypes`."""
    if t is not None and t.shape == shape and t.dtype in dtypes:
        return
    if t is None:
        raise ValueError(f"{name} is required")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}; expected one of {[str(d) for d in dtypes]}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}; expected {tuple(shape)}")


def _act_dtypes():
    torch = _torch()
    return (torch.float16, torch.bfloat16)


def _w4_group_count(K: int, group_size: int) -> int:
    if group_size <= 0 or K % group_size != 0:
        raise ValueError(f"K={K} is not a multiple of group_size={group_size}")
    return K // group_size


def _check_w4_weights(qweight, scales, qzeros, N, K, group_size, act, lead=()):
    """qweight [*lead, N, K/8] int32; scales [*lead, N, K/g] act; qzeros
    [*lead, N/8, K/g] int32 or None (activation-dtype zero-points are refused)."""
    torch = _torch()
    if K % 8 != 0 or N % 8 != 0:
        raise ValueError(f"K={K} and N={N} must be multiples of 8")
    G = _w4_group_count(K, group_size)
    _want(qweight, "qweight", (*lead, N, K // 8), (torch.int32,))
    _want(scales, "scales", (*lead, N, G), (act,))
    if qzeros is not None:
        if qzeros.dtype != torch.int32:
            raise TypeError(f"qzeros must be packed 4-bit zero-points (int32); dtype {qzeros.dtype} "
                            "is refused, not reinterpreted")
        _want(qzeros, "qzeros", (*lead, N // 8, G), (torch.int32,))


def device_check() -> None:
    """Raise unless the current device is gfx950."""
    _lib.check(_lib.lib().wob_device_check(), "device_check")


def gemm(x, qweight, scales, qzeros, group_size: int, out=None, path: int = PATH_AUTO):
    """W4A16 GEMM: y[M,N] = x[M,K] . ((q - z) * s)^T.

    x [M,K] fp16/bf16; qweight [N,K/8] int32; scales [N,K/g] x.dtype;
    qzeros [N/8,K/g] int32 (packed) or None (symmetric, z = 8); out [M,N] x.dtype.
    """
    torch = _torch()
    if x.dim() != 2 or qweight.dim() != 2:
        raise ValueError("x must be [M, K] and qweight [N, K/8]")
    _want(x, "x", tuple(x.shape), _act_dtypes())
    M, K = x.shape
    N = qweight.shape[0]
    _check_w4_weights(qweight, scales, qzeros, N, K, group_size, x.dtype)
    if out is None:
        out = torch.empty((M, N), dtype=x.dtype, device=x.device)
    _want(out, "out", (M, N), (x.dtype,))
    dev = _check_device(x, qweight, scales, qzeros, out)
    st = _run(_lib.lib().w4a16_gemm_ex, dev, _ptr(x), _tag(x), _ptr(qweight), _ptr(scales),
               _tag(scales), _ptr(qzeros), _tag(qzeros) if qzeros is not None else U4X8_I32,
               _ptr(out), M, N, K, group_size, path)
    _lib.check(st, "w4a16_gemm")
    return out


def gemm_grouped(x, m_offsets, qweight, scales, qzeros, group_size: int, out=None):
    """Ragged grouped W4A16 GEMM: x [total_M,K]; m_offsets device int64 [E+1];
    qweight [E,N,K/8] int32; scales [E,N,K/g]; qzeros [E,N/8,K/g] int32 or None;
    out [total_M,N] x.dtype."""
    torch = _torch()
    if x.dim() != 2 or qweight.dim() != 3:
        raise ValueError("x must be [total_M, K] and qweight [E, N, K/8]")
    _want(x, "x", tuple(x.shape), _act_dtypes())
    total_m, K = x.shape
    E, N = qweight.shape[0], qweight.shape[1]
    _check_w4_weights(qweight, scales, qzeros, N, K, group_size, x.dtype, lead=(E,))
    _want(m_offsets, "m_offsets", (E + 1,), (torch.int64,))
    if out is None:
        out = torch.empty((total_m, N), dtype=x.dtype, device=x.device)
    _want(out, "out", (total_m, N), (x.dtype,))
    dev = _check_device(x, m_offsets, qweight, scales, qzeros, out)
    st = _run(_lib.lib().w4a16_gemm_grouped, dev, _ptr(x), _tag(x), _ptr(m_offsets), E, total_m,
               _ptr(qweight), _ptr(scales), _tag(scales), _ptr(qzeros), _tag(qzeros) if qzeros is
               not None else U4X8_I32, _ptr(out), N, K, group_size)
    _lib.check(st, "w4a16_gemm_grouped")
    return out


def moe_workspace_size(T: int, topk: int, E: int, N: int = 0, K: int = 0) -> int:
    """Bytes of workspace mxfp4_moe_gemm needs (0 for arguments it refuses)."""
    return int(_lib.lib().mxfp4_moe_gemm_workspace_size(T, topk, E, N, K))


def mxfp4_moe_gemm(x, topk_ids, w_fp4, w_scale, out=None, workspace=None, act: int = ACT_NONE,
                   tile_m: int = 32):
    """MoE stage 1: x [T,K] bf16, topk_ids [T,topk] int32, w_fp4 [E,N,K/2] uint8 and
    w_scale [E,N,K/32] uint8 (E8M0) -> y [T,topk,N] bf16 (act=ACT_NONE) or
    y [T,topk,N/2] = silu(gate) * up (act=ACT_SILU_MUL).  workspace: device memory of
    at least moe_workspace_size(T, topk, E, N, K) bytes (allocated when None).
    tile_m: 32 (the default, mxfp4_moe_gemm) or 16 (mxfp4_moe_gemm_tile_m), the
    row padding of each expert's tile."""
    torch = _torch()
    if x.dim() != 2 or topk_ids.dim() != 2 or w_fp4.dim() != 3:
        raise ValueError("x must be [T, K], topk_ids [T, topk] and w_fp4 [E, N, K/2]")
    _want(x, "x", tuple(x.shape), (torch.bfloat16,))
    T, K = x.shape
    topk = topk_ids.shape[1]
    E, N = w_fp4.shape[0], w_fp4.shape[1]
    if K % 32 != 0:
        raise ValueError(f"K={K} must be a multiple of 32 (one E8M0 scale per 32)")
    _want(topk_ids, "topk_ids", (T, topk), (torch.int32,))
    _want(w_fp4, "w_fp4", (E, N, K // 2), (torch.uint8,))
    _want(w_scale, "w_scale", (E, N, K // 32), (torch.uint8,))
    if act not in (ACT_NONE, ACT_SILU_MUL):
        raise ValueError(f"unknown activation {act}")
    if tile_m not in (16, 32):
        raise ValueError(f"tile_m={tile_m} must be 16 or 32")
    nout = N // 2 if act == ACT_SILU_MUL else N
    if out is None:
        out = torch.empty((T, topk, nout), dtype=torch.bfloat16, device=x.device)
    _want(out, "out", (T, topk, nout), (torch.bfloat16,))
    need = moe_workspace_size(T, topk, E, N, K)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=x.device)
    ws_bytes = workspace.numel() * workspace.element_size()
    if ws_bytes < need:
        raise ValueError(f"workspace holds {ws_bytes} bytes; {need} are needed")
    dev = _check_device(x, topk_ids, w_fp4, w_scale, out, workspace)
    args = (_ptr(x), _ptr(topk_ids), _ptr(w_fp4), _ptr(w_scale), _ptr(out), T, topk, E, N, K, act)
    if tile_m == 32:
        st = _run(_lib.lib().mxfp4_moe_gemm, dev, *args, _ptr(workspace), ws_bytes)
    else:
        st = _run(_lib.lib().mxfp4_moe_gemm_tile_m, dev, *args, tile_m, _ptr(workspace), ws_bytes)
    _lib.check(st, "mxfp4_moe_gemm")
    return out


def moe_stage2_workspace_size(T: int, topk: int, E: int, H: int, I: int) -> int:
    """Bytes of workspace mxfp4_moe_stage2 needs (0 for arguments it refuses)."""
    return int(_lib.lib().mxfp4_moe_stage2_workspace_size(T, topk, E, H, I))


def mxfp4_moe_stage2(a, topk_ids, topk_weights, w2_fp4, w2_scale, out=None, workspace=None):
    """MoE stage 2: a [T,topk,I] bf16 (the stage-1 activation rows), topk_ids
    [T,topk] int32, topk_weights [T,topk] float32, w2_fp4 [E,H,I/2] uint8,
    w2_scale [E,H,I/32] uint8 (E8M0) -> y [T,H] bf16 = sum over slots of
    weight * (a row . expert's W2)."""
    torch = _torch()
    if a.dim() != 3 or topk_ids.dim() != 2 or w2_fp4.dim() != 3:
        raise ValueError("a must be [T, topk, I], topk_ids [T, topk] and w2_fp4 [E, H, I/2]")
    _want(a, "a", tuple(a.shape), (torch.bfloat16,))
    T, topk, I = a.shape
    E, H = w2_fp4.shape[0], w2_fp4.shape[1]
    if I % 32 != 0:
        raise ValueError(f"I={I} must be a multiple of 32 (one E8M0 scale per 32)")
    _want(topk_ids, "topk_ids", (T, topk), (torch.int32,))
    _want(topk_weights, "topk_weights", (T, topk), (torch.float32,))
    _want(w2_fp4, "w2_fp4", (E, H, I // 2), (torch.uint8,))
    _want(w2_scale, "w2_scale", (E, H, I // 32), (torch.uint8,))
    if out is None:
        out = torch.empty((T, H), dtype=torch.bfloat16, device=a.device)
    _want(out, "out", (T, H), (torch.bfloat16,))
    need = moe_stage2_workspace_size(T, topk, E, H, I)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=a.device)
    ws_bytes = workspace.numel() * workspace.element_size()
    if ws_bytes < need:
        raise ValueError(f"workspace holds {ws_bytes} bytes; {need} are needed")
    dev = _check_device(a, topk_ids, topk_weights, w2_fp4, w2_scale, out, workspace)
    st = _run(_lib.lib().mxfp4_moe_stage2, dev, _ptr(a), _ptr(topk_ids), _ptr(topk_weights),
               _ptr(w2_fp4), _ptr(w2_scale), _ptr(out), T, topk, E, H, I, _ptr(workspace), ws_bytes)
    _lib.check(st, "mxfp4_moe_stage2")
    return out


def _output(t, name, shape, dtype, device):
    """A caller's output on `device`, checked, or a new one, which needs no check."""
    if t is None:
        index = device.index  # None: the host, which the caller refuses
        if index is not None and len(shape) <= 2 and 0 not in shape and _get_device() == index:
            return _empty_here(shape, (shape[1], 1) if len(shape) == 2 else (1,) * len(shape), dtype)
        return _torch_mod.empty(shape, dtype=dtype, device=device)
    _want(t, name, shape, (dtype,))
    if _check_device(t) != device:
        raise ValueError("operands live on different devices")
    return t


def _workspace(workspace, need, device):
    """A caller's workspace, checked, or a new one where one is needed: (tensor, bytes)."""
    torch = _torch()
    if workspace is None:
        if need == 0:
            return None, 0
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    ws_bytes = workspace.numel() * workspace.element_size()
    if ws_bytes < need:
        raise ValueError(f"workspace holds {ws_bytes} bytes; {need} are needed")
    return workspace, ws_bytes


def mxfp4_quantize(x, out=None, out_scale=None):
    """MXFP4 quantisation along the last dimension: x [..., K] fp16/bf16/fp32 ->
    (codes [..., K/2] uint8, scale [..., K/32] uint8 E8M0), the layout the MXFP4
    products read.  x is contiguous, or 2-D with contiguous elements in each row
    and rows any 16-byte aligned distance apart (a column slice)."""
    torch = _torch()
    if x.dim() < 1:
        raise ValueError("x must be [..., K]")
    _want(x, "x", x.shape, _values)
    K = x.shape[-1]
    if K < 32 or K % 32 != 0:
        raise ValueError(f"K={K} must be a multiple of 32 (one E8M0 scale per 32)")
    lead = tuple(x.shape[:-1])
    R = 1
    for n in lead:
        R *= n
    if x.is_contiguous():
        ldx = K
    elif x.dim() == 2 and x.stride(1) == 1 and x.stride(0) >= K:
        ldx = x.stride(0)
    else:
        raise ValueError("x must be contiguous, or a 2-D column slice of a contiguous tensor")
    dev = x.device
    out = _output(out, "out", (*lead, K // 2), torch.uint8, dev)
    out_scale = _output(out_scale, "out_scale", (*lead, K // 32), torch.uint8, dev)
    if x.get_device() < 0:
        raise ValueError("all operands must be device tensors")
    st = _run(_lib.lib().mxfp4_quantize, dev, x.data_ptr(), _tags[x.dtype], ldx, out.data_ptr(),
               out_scale.data_ptr(), R, K)
    _lib.check(st, "mxfp4_quantize")
    return out, out_scale


@functools.lru_cache(maxsize=256)
def mxfp4_gemm_workspace_size(M: int, N: int, K: int) -> int:
    """Bytes of workspace mxfp4_gemm needs (0 also for arguments it refuses)."""
    return int(_lib.lib().mxfp4_gemm_workspace_size(M, N, K))


def mxfp4_gemm(x_fp4, x_scale, w_fp4, w_scale, out=None, out_dtype=None, workspace=None):
    """MXFP4 x MXFP4 product: x_fp4 [M,K/2], x_scale [M,K/32], w_fp4 [N,K/2] and
    w_scale [N,K/32] uint8 -> y [M,N] = x . w^T in out_dtype (bfloat16 when
    neither it nor out is given; float16 and float32 too)."""
    torch = _torch()
    if x_fp4.dim() != 2 or w_fp4.dim() != 2:
        raise ValueError("x_fp4 must be [M, K/2] and w_fp4 [N, K/2]")
    M, K = x_fp4.shape[0], x_fp4.shape[1] * 2
    N = w_fp4.shape[0]
    if K < 32 or K % 32 != 0:
        raise ValueError(f"K={K} must be a multiple of 32 (one E8M0 scale per 32)")
    _want(x_fp4, "x_fp4", (M, K // 2), _bytes)
    _want(x_scale, "x_scale", (M, K // 32), _bytes)
    _want(w_fp4, "w_fp4", (N, K // 2), _bytes)
    _want(w_scale, "w_scale", (N, K // 32), _bytes)
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else torch.bfloat16
    if out_dtype not in _values:
        raise TypeError(f"out_dtype {out_dtype} must be float16, bfloat16 or float32")
    dev = x_fp4.device
    out = _output(out, "out", (M, N), out_dtype, dev)
    workspace, ws_bytes = _workspace(workspace, mxfp4_gemm_workspace_size(M, N, K), dev)
    _check_device(x_fp4, x_scale, w_fp4, w_scale, workspace)
    st = _run(_lib.lib().mxfp4_gemm, dev, x_fp4.data_ptr(), x_scale.data_ptr(), w_fp4.data_ptr(),
               w_scale.data_ptr(), out.data_ptr(), _tags[out_dtype], M, N, K, _ptr(workspace), ws_bytes)
    _lib.check(st, "mxfp4_gemm")
    return out


def _check_choice(logits, topk, bias):
    """logits [T, E], bias [E] or None -> (T, E)."""
    torch = _torch()
    if logits.dim() != 2:
        raise ValueError("logits must be [T, E]")
    _want(logits, "logits", logits.shape, _values)
    T, E = logits.shape
    if not 1 <= topk <= min(E, 64):
        raise ValueError(f"topk={topk} must be between 1 and min(E={E}, 64)")
    if bias is not None:
        _want(bias, "bias", (E,), (torch.float32,))
    return T, E


def moe_topk(logits, topk: int, bias=None, renormalize: bool = True, ids=None, weights=None):
    """Choice of experts: logits [T,E] fp16/bf16/fp32 (+ bias [E] float32) ->
    (ids [T,topk] int32, weights [T,topk] float32), largest first, ties to the
    lowest expert.  weights: softmax over the chosen (renormalize) or over all
    experts.  Places without an expert above -inf hold id -1 and weight 0."""
    torch = _torch()
    T, E = _check_choice(logits, topk, bias)
    dev = logits.device
    ids = _output(ids, "ids", (T, topk), torch.int32, dev)
    weights = _output(weights, "weights", (T, topk), torch.float32, dev)
    _check_device(logits, bias)
    st = _run(_lib.lib().moe_topk, dev, logits.data_ptr(), _tags[logits.dtype], _ptr(bias),
               ids.data_ptr(), weights.data_ptr(), T, E, topk, 1 if renormalize else 0)
    _lib.check(st, "moe_topk")
    return ids, weights


@functools.lru_cache(maxsize=256)
def moe_layer_workspace_size(T: int, topk: int, E: int, H: int, I: int) -> int:
    """Bytes of workspace mxfp4_moe_layer needs (0 for arguments it refuses)."""
    return int(_lib.lib().mxfp4_moe_layer_workspace_size(T, topk, E, H, I))


def mxfp4_moe_layer(x, logits, topk: int, w1_fp4, w1_scale, w2_fp4, w2_scale, bias=None,
                    renormalize: bool = True, out=None, workspace=None):
    """A whole MoE layer from the router's scores: x [T,H] bf16, logits [T,E]
    (bias [E]) as for moe_topk, w1_fp4 [E,2I,H/2], w1_scale [E,2I,H/32], w2_fp4
    [E,H,I/2], w2_scale [E,H,I/32] uint8 -> y [T,H] bf16 = sum over the chosen
    experts of weight * W2(silu(W1g x) * (W1u x))."""
    torch = _torch()
    if x.dim() != 2 or w1_fp4.dim() != 3 or w2_fp4.dim() != 3:
        raise ValueError("x must be [T, H], w1_fp4 [E, 2I, H/2] and w2_fp4 [E, H, I/2]")
    T, E = _check_choice(logits, topk, bias)
    H, I = x.shape[1], w2_fp4.shape[2] * 2
    if H < 64 or I < 64 or H % 64 != 0 or I % 64 != 0:
        raise ValueError(f"H={H} and I={I} must be multiples of 64")
    _want(x, "x", (T, H), (torch.bfloat16,))
    _want(w1_fp4, "w1_fp4", (E, 2 * I, H // 2), _bytes)
    _want(w1_scale, "w1_scale", (E, 2 * I, H // 32), _bytes)
    _want(w2_fp4, "w2_fp4", (E, H, I // 2), _bytes)
    _want(w2_scale, "w2_scale", (E, H, I // 32), _bytes)
    dev = x.device
    out = _output(out, "out", (T, H), torch.bfloat16, dev)
    workspace, ws_bytes = _workspace(workspace, moe_layer_workspace_size(T, topk, E, H, I), dev)
    _check_device(x, logits, bias, w1_fp4, w1_scale, w2_fp4, w2_scale, workspace)
    st = _run(_lib.lib().mxfp4_moe_layer, dev, x.data_ptr(), logits.data_ptr(), _tags[logits.dtype],
               _ptr(bias), w1_fp4.data_ptr(), w1_scale.data_ptr(), w2_fp4.data_ptr(),
               w2_scale.data_ptr(), out.data_ptr(), T, topk, E, H, I, 1 if renormalize else 0,
               _ptr(workspace), ws_bytes)
    _lib.check(st, "mxfp4_moe_layer")
    return out


# The operators below are called for single tokens, where the host's time is the call's: their
# operands are checked in one pass each, outputs made on the current device, and a call for another
# device is made again with that one current.

def _operand(t, name, shape, dtypes, index):
    """_want, and t is contiguous and lives where the call's first operand does (index: its
    get_device(), below 0 for the host, which is refused once all shapes are right)."""
    if t is None or t.shape != shape or t.dtype not in dtypes:
        _want(t, name, shape, dtypes)
    if not t.is_contiguous():
        raise ValueError("all operands must be contiguous")
    if t.get_device() != index:
        raise ValueError("operands live on different devices")


def _elsewhere(index):
    """Whether the call has to be made again with device `index` current."""
    if index < 0:
        raise ValueError("all operands must be device tensors")
    return _get_device() != index


def _library():
    global _loaded
    _loaded = _lib.lib()
    return _loaded


def _contiguous_strides(shape):
    if len(shape) == 2:
        return (shape[1] or 1, 1)
    if len(shape) == 1:
        return (1,)
    strides, n = [], 1
    for d in reversed(shape):
        strides.append(n)
        n *= max(d, 1)
    return tuple(reversed(strides))


def _row_stride(x, name):
    """Elements from one row of x [..., K] to the next: x is contiguous, or 2-D with
    contiguous elements in each row (a column slice)."""
    K = x.shape[-1]
    if x.is_contiguous():
        return K
    if x.dim() == 2 and x.stride(1) == 1 and x.stride(0) >= K:
        return x.stride(0)
    raise ValueError(f"{name} must be contiguous, or a 2-D column slice of a contiguous tensor")


def _rows_like(t, name, shape, dtypes, index):
    """_operand for rows that may be a column slice; elements from one row to the next."""
    if t.shape != shape or t.dtype not in dtypes:
        _want(t, name, shape, dtypes)
    if t.get_device() != index:
        raise ValueError("operands live on different devices")
    return _row_stride(t, name)


def int8_quantize(x, act: int = ACT_NONE, out=None, out_scale=None):
    """Rows in 8 bits: x [..., K] fp16/bf16/fp32 -> (codes [..., K] int8, scale [...]
    float32), scale = amax / 127 of each row, the operands of int8_gemm.  act=ACT_SILU_MUL:
    x [..., 2K] holds gate and up halves, and silu(gate) * up is quantised.  x is
    contiguous, or 2-D with contiguous elements in each row and rows any 16-byte aligned
    distance apart (a column slice)."""
    torch = _torch_mod or _torch()
    shape = tuple(x.shape)
    if not shape:
        raise ValueError("x must be [..., K]")
    tag = _value_tags.get(x.dtype)
    if tag is None:
        _want(x, "x", shape, _values)
    K = shape[-1]
    if act == ACT_SILU_MUL:
        if K % 2 != 0:
            raise ValueError(f"x has {K} columns; gate and up halves make an even number")
        K //= 2
        shape = (*shape[:-1], K)
    elif act != ACT_NONE:
        raise ValueError(f"unknown activation {act}")
    if not 16 <= K <= 65536 or K % 16 != 0:
        raise ValueError(f"K={K} must be a multiple of 16, up to 65536")
    lead, ldx, index = shape[:-1], _row_stride(x, "x"), x.get_device()
    if out is not None:
        _operand(out, "out", shape, _int8, index)
    if out_scale is not None:
        _operand(out_scale, "out_scale", lead, _fp32, index)
    if _elsewhere(index):
        with torch.cuda.device(index):
            return int8_quantize(x, act, out, out_scale)
    if out is None:
        out = _empty_here(shape, _contiguous_strides(shape), torch.int8)
    if out_scale is None:
        out_scale = _empty_here(lead, _contiguous_strides(lead), torch.float32)
    st = (_loaded or _library()).int8_quantize(
        x.data_ptr(), tag, ldx, act, out.data_ptr(), out_scale.data_ptr(), out.numel() // K, K,
        _raw_stream(index))
    if st:
        _lib.check(st, "int8_quantize")
    return out, out_scale


def int8_dequant(codes, scale, out_dtype=None, out=None):
    """Rows in 8 bits read back: codes [..., K] int8 and scale [...] float32 -> values
    [..., K] in out_dtype (bfloat16 when neither it nor out is given)."""
    torch = _torch_mod or _torch()
    shape, index = tuple(codes.shape), codes.get_device()
    if not shape:
        raise ValueError("codes must be [..., K]")
    lead, K = shape[:-1], shape[-1]
    _operand(codes, "codes", shape, _int8, index)
    if not 16 <= K <= 65536 or K % 16 != 0:
        raise ValueError(f"K={K} must be a multiple of 16, up to 65536")
    _operand(scale, "scale", lead, _fp32, index)
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else torch.bfloat16
    tag = _value_tags.get(out_dtype)
    if tag is None:
        raise TypeError(f"out_dtype {out_dtype} must be float16, bfloat16 or float32")
    if out is not None:
        _operand(out, "out", shape, (out_dtype,), index)
    if _elsewhere(index):
        with torch.cuda.device(index):
            return int8_dequant(codes, scale, out_dtype, out)
    if out is None:
        out = _empty_here(shape, _contiguous_strides(shape), out_dtype)
    st = (_loaded or _library()).int8_dequant(codes.data_ptr(), scale.data_ptr(), out.data_ptr(), tag,
                                              out.numel() // K, K, _raw_stream(index))
    if st:
        _lib.check(st, "int8_dequant")
    return out


@functools.lru_cache(maxsize=256)
def int8_gemm_workspace_size(M: int, N: int, K: int) -> int:
    """Bytes of workspace int8_gemm needs (0 also for arguments it refuses)."""
    return int(_lib.lib().int8_gemm_workspace_size(M, N, K))


def int8_gemm(x_q, x_scale, w_q, w_scale, bias=None, out=None, out_dtype=None, workspace=None):
    """8-bit product: x_q [M,K] int8 with x_scale [M] float32 (a token's), w_q [N,K] int8
    with w_scale [N] float32 (a channel's) -> y [M,N] = x_scale * w_scale * (x_q . w_q^T)
    (+ bias [N] float32) in out_dtype (bfloat16 when neither it nor out is given; float16
    and float32 too).  The sum over K is exact."""
    torch = _torch_mod or _torch()
    if x_q.dim() != 2 or w_q.dim() != 2:
        raise ValueError("x_q must be [M, K] and w_q [N, K]")
    M, K = x_q.shape
    N = w_q.shape[0]
    index = x_q.get_device()
    _operand(x_q, "x_q", (M, K), _int8, index)
    _operand(x_scale, "x_scale", (M,), _fp32, index)
    _operand(w_q, "w_q", (N, K), _int8, index)
    _operand(w_scale, "w_scale", (N,), _fp32, index)
    if bias is not None:
        _operand(bias, "bias", (N,), _fp32, index)
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else torch.bfloat16
    tag = _value_tags.get(out_dtype)
    if tag is None:
        raise TypeError(f"out_dtype {out_dtype} must be float16, bfloat16 or float32")
    if out is not None:
        _operand(out, "out", (M, N), (out_dtype,), index)
    if _elsewhere(index):
        with torch.cuda.device(index):
            return int8_gemm(x_q, x_scale, w_q, w_scale, bias, out, out_dtype, workspace)
    need = ws_bytes = int8_gemm_workspace_size(M, N, K)
    if workspace is not None:
        workspace, ws_bytes = _workspace(workspace, need, x_q.device)
        _check_device(x_q, workspace)
    elif need:
        workspace = _empty_here((need,), (1,), torch.uint8)
    if out is None:
        out = _empty_here((M, N), (max(N, 1), 1), out_dtype)
    st = (_loaded or _library()).int8_gemm(
        x_q.data_ptr(), x_scale.data_ptr(), w_q.data_ptr(), w_scale.data_ptr(), _ptr(bias), out.data_ptr(),
        tag, M, N, K, _ptr(workspace), ws_bytes, _raw_stream(index))
    if st:
        _lib.check(st, "int8_gemm")
    return out


def residual_norm(y, residual, weight, post_weight=None, gate=None, alpha: float = 1.0,
                  eps: float = 1e-6, quant: int = QUANT_NONE, out=None, out_scale=None,
                  residual_out=None):
    """The norms after a block and before the next, with its gate and residual scale:

        t = y, or y / rms(y) * post_weight;  h = residual + alpha * gate * t
        n = h / rms(h) * weight,             rms(v) = sqrt(mean(v^2) + eps)

    y [T,H] fp16/bf16/fp32 (contiguous or a column slice); residual [T,H] in y's dtype
    or float32; weight, post_weight [H]; gate [H] or [T,H] (contiguous or a column slice).
    Returns (n, h) with h in residual's dtype and n in y's, or (codes, scale, h) with
    quant=QUANT_INT8 (as int8_quantize) or QUANT_MXFP4 (as mxfp4_quantize).  residual_out
    may be residual itself.  y=None: n of the residual alone (then h is residual, and n has
    weight's dtype).  weight=None: no n (it is returned as None)."""
    torch = _torch_mod or _torch()
    if residual.dim() != 2:
        raise ValueError("residual must be [T, H]")
    T, H = shape = tuple(residual.shape)
    block = y if y is not None else weight
    if block is None:
        raise ValueError("y and weight are both missing: there is nothing to compute")
    dt, rdt = block.dtype, residual.dtype
    tag = _value_tags.get(dt)
    if tag is None:
        raise TypeError(f"dtype {dt} must be float16, bfloat16 or float32")
    own = (dt,)
    index = residual.get_device()
    _operand(residual, "residual", shape, own if rdt == dt else _fp32, index)
    whole = 8 if quant == QUANT_NONE else 16 if quant == QUANT_INT8 else 32
    if whole == 32 and quant != QUANT_MXFP4:
        raise ValueError(f"unknown quant {quant}")
    if not whole <= H <= 32768 or H % whole != 0:
        raise ValueError(f"H={H} must be a multiple of {whole}, up to 32768")
    if not (math.isfinite(alpha) and math.isfinite(eps) and eps >= 0):
        raise ValueError(f"alpha={alpha} must be finite, eps={eps} finite and not negative")
    ldy = ldg = 0
    if y is not None:
        ldy = _rows_like(y, "y", shape, own, index)
        if post_weight is not None:
            _operand(post_weight, "post_weight", (H,), own, index)
        if gate is not None:
            if gate.dim() == 1:
                _operand(gate, "gate", (H,), own, index)
            else:
                ldg = _rows_like(gate, "gate", shape, own, index)
        if residual_out is not None and residual_out is not residual:
            _operand(residual_out, "residual_out", shape, (rdt,), index)
    elif post_weight is not None or gate is not None:
        raise ValueError("without y there is no post_weight and no gate")
    elif residual_out is not None:
        raise ValueError("without y the residual does not change: residual_out must be None")
    if weight is None:
        if quant != QUANT_NONE or out is not None or out_scale is not None:
            raise ValueError("without weight there are no normed rows")
    else:
        _operand(weight, "weight", (H,), own, index)
        if quant == QUANT_NONE:
            if out_scale is not None:
                raise ValueError("out_scale without quantised rows")
            width, kind = H, dt
        elif quant == QUANT_INT8:
            width, kind = H, torch.int8
            if out_scale is not None:
                _operand(out_scale, "out_scale", (T,), _fp32, index)
        else:
            width, kind = H // 2, torch.uint8
            if out_scale is not None:
                _operand(out_scale, "out_scale", (T, H // 32), _bytes, index)
        if out is not None:
            _operand(out, "out", (T, width), (kind,), index)
    if _elsewhere(index):
        with torch.cuda.device(index):
            return residual_norm(y, residual, weight, post_weight, gate, alpha, eps, quant, out, out_scale,
                                 residual_out)
    if y is not None and residual_out is None:
        residual_out = _empty_here(shape, (H, 1), rdt)
    if weight is not None:
        if out is None:
            out = _empty_here((T, width), (width, 1), kind)
        if out_scale is None and quant != QUANT_NONE:
            out_scale = (_empty_here((T,), (1,), torch.float32) if quant == QUANT_INT8 else
                         _empty_here((T, H // 32), (H // 32, 1), torch.uint8))
    st = (_loaded or _library()).residual_norm(
        _ptr(y), tag, ldy, residual.data_ptr(), _value_tags[rdt], _ptr(post_weight), _ptr(gate), ldg, alpha,
        _ptr(weight), eps, quant, _ptr(out), _ptr(out_scale), _ptr(residual_out), T, H, _raw_stream(index))
    if st:
        _lib.check(st, "residual_norm")
    h = residual if y is None else residual_out
    return (out, h) if quant == QUANT_NONE else (out, out_scale, h)


def moe_route(logits, topk: int, bias=None, score: int = SCORE_SIGMOID, groups: int = 1,
              topk_groups: int = 1, group_top: int = 2, renormalize: bool = True,
              scale: float = 1.0, ids=None, weights=None):
    """Group-limited choice of experts: logits [T,E] fp16/bf16/fp32 -> (ids [T,topk] int32,
    weights [T,topk] float32), what the MoE stages take.  Scores s: sigmoid of the logits,
    or their softmax over all experts.  The choice goes by s + bias (bias [E] float32): the
    topk_groups groups with the largest sum of their group_top (1 or 2) best, then the topk
    best experts in them, ties to the lowest index.  weights: scale * s, over the chosen
    experts' sum with renormalize.  Places without an expert hold id -1 and weight 0."""
    torch = _torch_mod or _torch()
    if logits.dim() != 2:
        raise ValueError("logits must be [T, E]")
    T, E = shape = tuple(logits.shape)
    index = logits.get_device()
    _operand(logits, "logits", shape, _values, index)
    if score not in (SCORE_SIGMOID, SCORE_SOFTMAX):
        raise ValueError(f"unknown score {score}")
    if not 1 <= groups <= 64 or not 1 <= E <= 1024 or E % groups != 0:
        raise ValueError(f"E={E} (up to 1024) must be a multiple of groups={groups} (up to 64)")
    if not 1 <= topk_groups <= groups:
        raise ValueError(f"topk_groups={topk_groups} must be between 1 and groups={groups}")
    if not 1 <= topk <= 64 or topk > topk_groups * (E // groups):
        raise ValueError(f"topk={topk} must be between 1 and 64 and at most the kept groups' experts")
    if group_top not in (1, 2):
        raise ValueError(f"group_top={group_top} must be 1 or 2")
    if bias is not None:
        _operand(bias, "bias", (E,), _fp32, index)
    if ids is not None:
        _operand(ids, "ids", (T, topk), (torch.int32,), index)
    if weights is not None:
        _operand(weights, "weights", (T, topk), _fp32, index)
    if _elsewhere(index):
        with torch.cuda.device(index):
            return moe_route(logits, topk, bias, score, groups, topk_groups, group_top, renormalize, scale,
                             ids, weights)
    if ids is None:
        ids = _empty_here((T, topk), (topk, 1), torch.int32)
    if weights is None:
        weights = _empty_here((T, topk), (topk, 1), torch.float32)
    st = (_loaded or _library()).moe_route(
        logits.data_ptr(), _value_tags[logits.dtype], _ptr(bias), ids.data_ptr(), weights.data_ptr(), T, E, topk,
        score, groups, topk_groups, group_top, 1 if renormalize else 0, scale, _raw_stream(index))
    if st:
        _lib.check(st, "moe_route")
    return ids, weights


def w4a16_dequant(qweight, scales, qzeros, group_size: int, out_dtype=None):
    """Probe: the kernels' dequantized weights [N,K] (float32 skinny form, or
    the scales' dtype for the MFMA operand form)."""
    torch = _torch()
    if qweight.dim() != 2:
        raise ValueError("qweight must be [N, K/8]")
    N, K = qweight.shape[0], qweight.shape[1] * 8
    if scales.dtype not in _act_dtypes():
        raise TypeError(f"scales must be float16 or bfloat16, not {scales.dtype}")
    _check_w4_weights(qweight, scales, qzeros, N, K, group_size, scales.dtype)
    out_dtype = out_dtype or torch.float32
    if out_dtype not in (torch.float32, scales.dtype):
        raise TypeError("out_dtype must be float32 or the scales' dtype")
    out = torch.empty((N, K), dtype=out_dtype, device=qweight.device)
    dev = _check_device(qweight, scales, qzeros, out)
    st = _run(_lib.lib().w4a16_dequant, dev, _ptr(qweight), _ptr(scales), _tag(scales),
               _ptr(qzeros), _tag(qzeros) if qzeros is not None else U4X8_I32, _ptr(out), _tag(out),
               N, K, group_size)
    _lib.check(st, "w4a16_dequant")
    return out


def mxfp4_dequant(w_fp4, w_scale):
    """Probe: the MoE kernels' bf16 weight-operand values [N,K] for one expert."""
    torch = _torch()
    if w_fp4.dim() != 2:
        raise ValueError("w_fp4 must be [N, K/2]")
    N, K = w_fp4.shape[0], w_fp4.shape[1] * 2
    if K % 32 != 0:
        raise ValueError(f"K={K} must be a multiple of 32")
    _want(w_fp4, "w_fp4", (N, K // 2), _bytes)
    _want(w_scale, "w_scale", (N, K // 32), _bytes)
    out = torch.empty((N, K), dtype=torch.bfloat16, device=w_fp4.device)
    dev = _check_device(w_fp4, w_scale, out)
    st = _run(_lib.lib().mxfp4_dequant, dev, _ptr(w_fp4), _ptr(w_scale), _ptr(out), N, K)
    _lib.check(st, "mxfp4_dequant")
    return out


def stream_read(buf, nbytes: int, sink) -> None:
    """Measurement aid: read nbytes of the device tensor buf once (the device's
    streaming-read reference for a byte count); sink: >= 1024 bytes of scratch."""
    torch = _torch()
    if nbytes > buf.numel() * buf.element_size() or sink.numel() * sink.element_size() < 1024:
        raise ValueError("buffer smaller than nbytes or sink under 1024 bytes")
    dev = _check_device(buf, sink)
    st = _run(_lib.lib().wob_stream_read, dev, _ptr(buf), nbytes, _ptr(sink))
    _lib.check(st, "wob_stream_read")
