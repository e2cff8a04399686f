"""The 8-bit operators of libdora_mi355x.so: the norm in front of an 8-bit
product, rows to 8 bits and back, the product itself, and their autograd
wiring.  Like binding.py, argument marshalling only.

A weight in 8 bits is (codes, scale): int8 [d_out, d_in] and fp32 [d_out], made
once with quantize_rows from the merged weight (or from a frozen W0).  An
activation in 8 bits is the same with a scale per token.
"""
from __future__ import annotations

import ctypes
import functools

import torch
from torch.autograd.function import once_differentiable

from .binding import _DTYPE_CODE, _call, _check, _extent, _need, load, workspace

_F32, _I8 = torch.float32, torch.int8
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)

# A decoding step's calls take a few microseconds on the GPU, no more than the
# host spends on one: arguments are compared in place, and pointers and the
# stream are passed as plain integers.


def _stream(device) -> int:
    """The current stream's handle (torch.cuda.current_stream builds an object for it)."""
    if device.type != "cuda":
        raise ValueError(f"tensors must be on a GPU (got {device})")
    return _raw_stream(device.index) if _raw_stream is not None else torch.cuda.current_stream(device).cuda_stream


def _matrix(t, name: str):
    """(device, dtype, shape) of a contiguous 2-D float tensor."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} has shape {tuple(shape)}, expected two dimensions")
    if t.dtype not in _DTYPE_CODE:
        raise ValueError(f"unsupported dtype {t.dtype} of {name}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.device, t.dtype, shape


def _in(t, name: str, device, dtype, shape) -> int:
    """The pointer of an argument that has to be this; _need says what it is not."""
    if not isinstance(t, torch.Tensor) or t.shape != shape or t.dtype != dtype or t.device != device or \
            not t.is_contiguous():
        _need(t, name, device, dtype, shape)
    return t.data_ptr()


def _out(t, name: str, device, dtype, shape, like=None):
    """An output: the caller's, or a new one (like another tensor where there is one of its kind: that is quicker)."""
    if t is None:
        return torch.empty(*shape, dtype=dtype, device=device) if like is None else torch.empty_like(like)
    _in(t, name, device, dtype, shape)
    return t


@functools.lru_cache(maxsize=4096)
def rmsnorm_backward_workspace_size(T: int, d: int) -> int:
    n = ctypes.c_size_t(0)
    _check(load().dora_rmsnorm_backward_workspace_size(T, d, ctypes.byref(n)), "dora_rmsnorm_backward_workspace_size")
    return n.value


@functools.lru_cache(maxsize=4096)
def matmul_q8_workspace_size(T: int, d_out: int, d_in: int) -> int:
    n = ctypes.c_size_t(0)
    _check(load().dora_matmul_q8_workspace_size(T, d_out, d_in, ctypes.byref(n)), "dora_matmul_q8_workspace_size")
    return n.value


def _scratch(ws, nbytes: int, device):
    """(buffer, pointer, bytes): the caller's workspace or the call's own, which the call holds."""
    if ws is not None:
        return (ws, *_extent(ws, device))
    ws = workspace(nbytes, device)
    return ws, None if ws is None else ws.data_ptr(), nbytes


# ------------------------------------------------------------ norm
def _norm(x, w, eps, residual, h, dev, dt, shape, y, q, scale, rstd):
    """The call, and h: x itself where there is no residual."""
    wp = _in(w, "w", dev, dt, shape[1:])
    rp = hp = None
    if residual is not None:
        rp = _in(residual, "residual", dev, dt, shape)
        h = _out(h, "h", dev, dt, shape, x)
        hp = h.data_ptr()
    elif h is not None:
        raise ValueError("h is an output of the addition: it needs a residual")
    _call("dora_rmsnorm", dev, x.data_ptr(), rp, wp, eps, shape[0], shape[1], _DTYPE_CODE[dt], hp,
          None if y is None else y.data_ptr(), None if q is None else q.data_ptr(),
          None if scale is None else scale.data_ptr(), None if rstd is None else rstd.data_ptr(), _stream(dev))
    return x if residual is None else h


def rmsnorm(x, w, eps: float, residual=None, *, y=None, h=None, rstd=None):
    """(y, h, rstd): h = x + residual, rstd = 1/sqrt(mean h^2 + eps) by rows, y = h rstd w.

    x, residual [T, d] and w [d] share a dtype (fp32, bf16 or fp16).  Without a
    residual h is x itself.  h=x or h=residual adds in place.
    """
    dev, dt, shape = _matrix(x, "x")
    y = _out(y, "y", dev, dt, shape, x)
    rstd = _out(rstd, "rstd", dev, _F32, shape[:1])
    h = _norm(x, w, eps, residual, h, dev, dt, shape, y, None, None, rstd)
    return y, h, rstd


def rmsnorm_q8(x, w, eps: float, residual=None, *, q=None, scale=None, h=None, y=None):
    """(q, scale, h): the norm's output in 8 bits with a scale per token, and h = x + residual.

    As rmsnorm, with y quantised before it is rounded.  y=tensor [T, d] also
    writes y itself (an unmerged adapter's branch reads it).
    """
    dev, dt, shape = _matrix(x, "x")
    q = _out(q, "q", dev, _I8, shape)
    scale = _out(scale, "scale", dev, _F32, shape[:1])
    if y is not None:
        _in(y, "y", dev, dt, shape)
    h = _norm(x, w, eps, residual, h, dev, dt, shape, y, q, scale, None)
    return q, scale, h


def rmsnorm_backward(dy, h, w, rstd, dh=None, *, need_dw: bool = True, dx=None, dw=None, ws=None):
    """(dx, dw) of rmsnorm's y (gradient dy) and h (gradient dh or None); dx is the
    gradient of x and of the residual, dw is fp32 [d] (None unless need_dw)."""
    dev, dt, shape = _matrix(dy, "dy")
    T, d = shape
    hp = _in(h, "h", dev, dt, shape)
    wp = _in(w, "w", dev, dt, shape[1:])
    rp = _in(rstd, "rstd", dev, _F32, shape[:1])
    dhp = None if dh is None else _in(dh, "dh", dev, dt, shape)
    dx = _out(dx, "dx", dev, dt, shape, dy)
    if need_dw:
        dw = _out(dw, "dw", dev, _F32, shape[1:])
        ws, wsp, nbytes = _scratch(ws, rmsnorm_backward_workspace_size(T, d), dev)
    else:
        dw, wsp, nbytes = None, None, 0
    _call("dora_rmsnorm_backward", dev, dy.data_ptr(), hp, wp, rp, dhp, T, d, _DTYPE_CODE[dt], dx.data_ptr(),
          None if dw is None else dw.data_ptr(), wsp, nbytes, _stream(dev))
    return dx, dw


# ------------------------------------------------------------ rows in 8 bits
def quantize_rows(x, col_scale=None, *, q=None, scale=None):
    """(q, scale): the rows of x * col_scale as int8 codes in [-127, 127] with an fp32 scale each."""
    dev, dt, shape = _matrix(x, "x")
    cp = None if col_scale is None else _in(col_scale, "col_scale", dev, _F32, shape[1:])
    q = _out(q, "q", dev, _I8, shape)
    scale = _out(scale, "scale", dev, _F32, shape[:1])
    _call("dora_quantize_rows", dev, x.data_ptr(), cp, shape[0], shape[1], _DTYPE_CODE[dt], q.data_ptr(),
          scale.data_ptr(), _stream(dev))
    return q, scale


def dequantize_rows(q, scale, dtype: torch.dtype, *, out=None):
    """q * scale by rows, rounded once to dtype."""
    dev, shape = _codes(q, "q")
    if dtype not in _DTYPE_CODE:
        raise ValueError(f"unsupported dtype {dtype}")
    sp = _in(scale, "scale", dev, _F32, shape[:1])
    out = _out(out, "out", dev, dtype, shape)
    _call("dora_dequantize_rows", dev, q.data_ptr(), sp, shape[0], shape[1], _DTYPE_CODE[dtype], out.data_ptr(),
          _stream(dev))
    return out


# ------------------------------------------------------------ product
def _codes(t, name: str):
    """(device, shape) of a contiguous 2-D int8 tensor."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    shape = t.shape
    if len(shape) != 2 or t.dtype != _I8 or not t.is_contiguous():
        raise ValueError(f"{name} must be int8, of two dimensions and contiguous (got {t.dtype}, {tuple(shape)})")
    return t.device, shape


def matmul_q8(xq, xscale, wq, wscale=None, dtype: torch.dtype = torch.bfloat16, *, bias=None, g=None, lora_out=None,
              s: float = 1.0, out=None, ws=None):
    """y = base + ((g-1) base + (g s) lora_out) + bias, base = xscale wscale (xq wq^T) with the sum exact.

    xq int8 [T, d_in] with xscale fp32 [T], wq int8 [d_out, d_in] with wscale
    fp32 [d_out] (None: ones).  g fp32 [d_out] with lora_out [T, d_out] of
    dtype, and bias fp32 [d_out], are optional.  y has dtype.
    """
    dev, (T, K) = _codes(xq, "xq")
    N = _codes(wq, "wq")[1][0]
    wp = _in(wq, "wq", dev, _I8, (N, K))
    if dtype not in _DTYPE_CODE:
        raise ValueError(f"unsupported dtype {dtype}")
    if (g is None) != (lora_out is None):
        raise ValueError("g and lora_out are given together or not at all")
    xsp = _in(xscale, "xscale", dev, _F32, (T,))
    wsp = None if wscale is None else _in(wscale, "wscale", dev, _F32, (N,))
    bp = None if bias is None else _in(bias, "bias", dev, _F32, (N,))
    gp = lp = None
    if g is not None:
        gp = _in(g, "g", dev, _F32, (N,))
        lp = _in(lora_out, "lora_out", dev, dtype, (T, N))
    out = _out(out, "out", dev, dtype, (T, N))
    ws, wkp, nbytes = _scratch(ws, matmul_q8_workspace_size(T, N, K), dev)
    _call("dora_matmul_q8", dev, xq.data_ptr(), xsp, wp, wsp, bp, gp, lp, s, T, N, K, _DTYPE_CODE[dtype],
          out.data_ptr(), wkp, nbytes, _stream(dev))
    return out


def linear_q8(x, wq, wscale, *, bias=None, g=None, lora_out=None, s: float = 1.0, out=None, ws=None):
    """matmul_q8 of x [T, d_in], quantised by rows here; y has x's dtype."""
    xq, xscale = quantize_rows(x)
    return matmul_q8(xq, xscale, wq, wscale, x.dtype, bias=bias, g=g, lora_out=lora_out, s=s, out=out, ws=ws)


def linear_q8_backward(dy, wqt, wscale, *, out=None, ws=None):
    """d_x of the linear map x -> x (wscale wq)^T, with dy * wscale quantised by rows.

    wqt int8 [d_in, d_out] is wq transposed, laid out once:
    wq.t().contiguous().
    """
    dq, dscale = quantize_rows(dy, wscale)
    return matmul_q8(dq, dscale, wqt, None, dy.dtype, out=out, ws=ws)


# ------------------------------------------------------------ autograd
class RMSNorm(torch.autograd.Function):
    """y, h = RMSNorm.apply(x, residual, w, eps); residual may be None, and then
    y alone is returned."""

    @staticmethod
    def forward(ctx, x, residual, w, eps):
        ctx.set_materialize_grads(False)
        y, h, rstd = rmsnorm(x, w, eps, residual)
        ctx.save_for_backward(h, w, rstd)
        ctx.has_residual = residual is not None
        return (y, h) if ctx.has_residual else y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh=None):
        h, w, rstd = ctx.saved_tensors
        if dy is None:   # only h was used
            return dh, dh, None, None
        dx, dw = rmsnorm_backward(dy.contiguous(), h, w, rstd, None if dh is None else dh.contiguous(),
                                  need_dw=ctx.needs_input_grad[2])
        return (dx, dx if ctx.has_residual else None, None if dw is None else dw.to(w.dtype), None)


class LinearQ8(torch.autograd.Function):
    """y = LinearQ8.apply(x, wq, wscale, wqt): a frozen weight in 8 bits in a
    training step.  The rounding of x and of dy passes gradients straight
    through: d_x is that of the linear map x -> x (wscale wq)^T."""

    @staticmethod
    def forward(ctx, x, wq, wscale, wqt):
        ctx.save_for_backward(wqt, wscale)
        return linear_q8(x, wq, wscale)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        wqt, wscale = ctx.saved_tensors
        return linear_q8_backward(dy.contiguous(), wqt, wscale), None, None, None
