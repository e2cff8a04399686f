"""The 8-bit operators of libdora_mi355x.so: the norm in front of an 8-bit
product, rows to 8 bits and back, the product itself, and their autograd
wiring.  Like binding.py, argument marshalling only.

A weight in 8 bits is (codes, scale): int8 [d_out, d_in] and fp32 [d_out], made
once with quantize_rows from the merged weight (or from a frozen W0).  An
activation in 8 bits is the same with a scale per token.
"""
from __future__ import annotations

import ctypes

import torch

from .binding import _DTYPE_CODE, _check, _need, _ptr, _stream, load, workspace

_F32, _I8 = torch.float32, torch.int8


def _rows(t, name: str):
    """(device, dtype, rows, row length) of a contiguous 2-D float tensor."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != 2:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected two dimensions")
    if t.dtype not in _DTYPE_CODE:
        raise ValueError(f"unsupported dtype {t.dtype} of {name}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.device, t.dtype, t.shape[0], t.shape[1]


def _out(t, name: str, device, dtype, shape):
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _need(t, name, device, dtype, shape)
    return t


def _nbytes(ws) -> int:
    return 0 if ws is None else ws.numel() * ws.element_size()


def rmsnorm_backward_workspace_size(T: int, d: int) -> int:
    n = ctypes.c_size_t(0)
    _check(load().dora_rmsnorm_backward_workspace_size(T, d, ctypes.byref(n)), "dora_rmsnorm_backward_workspace_size")
    return n.value


def matmul_q8_workspace_size(T: int, d_out: int, d_in: int) -> int:
    n = ctypes.c_size_t(0)
    _check(load().dora_matmul_q8_workspace_size(T, d_out, d_in, ctypes.byref(n)), "dora_matmul_q8_workspace_size")
    return n.value


# ------------------------------------------------------------ norm
def _norm(x, w, eps, residual, h, y, q, scale, rstd):
    dev, dt, T, d = _rows(x, "x")
    _need(w, "w", dev, dt, (d,))
    _check(load().dora_rmsnorm(_ptr(x), _ptr(residual), _ptr(w), float(eps), T, d, _DTYPE_CODE[dt], _ptr(h), _ptr(y),
                               _ptr(q), _ptr(scale), _ptr(rstd), _stream(dev)), "dora_rmsnorm")


def rmsnorm(x, w, eps: float, residual=None, *, y=None, h=None, rstd=None):
    """(y, h, rstd): h = x + residual, rstd = 1/sqrt(mean h^2 + eps) by rows, y = h rstd w.

    x, residual [T, d] and w [d] share a dtype (fp32, bf16 or fp16).  Without a
    residual h is x itself.  h=x or h=residual adds in place.
    """
    dev, dt, T, d = _rows(x, "x")
    y = _out(y, "y", dev, dt, (T, d))
    rstd = _out(rstd, "rstd", dev, _F32, (T,))
    if residual is not None:
        _need(residual, "residual", dev, dt, (T, d))
        h = _out(h, "h", dev, dt, (T, d))
    elif h is not None:
        raise ValueError("h is an output of the addition: it needs a residual")
    _norm(x, w, eps, residual, h, y, None, None, rstd)
    return y, (x if residual is None else h), rstd


def rmsnorm_q8(x, w, eps: float, residual=None, *, q=None, scale=None, h=None, y=None):
    """(q, scale, h): the norm's output in 8 bits with a scale per token, and h = x + residual.

    As rmsnorm, with y quantised before it is rounded.  y=tensor [T, d] also
    writes y itself (an unmerged adapter's branch reads it).
    """
    dev, dt, T, d = _rows(x, "x")
    q = _out(q, "q", dev, _I8, (T, d))
    scale = _out(scale, "scale", dev, _F32, (T,))
    if y is not None:
        _need(y, "y", dev, dt, (T, d))
    if residual is not None:
        _need(residual, "residual", dev, dt, (T, d))
        h = _out(h, "h", dev, dt, (T, d))
    elif h is not None:
        raise ValueError("h is an output of the addition: it needs a residual")
    _norm(x, w, eps, residual, h, y, q, scale, None)
    return q, scale, (x if residual is None else h)


def rmsnorm_backward(dy, h, w, rstd, dh=None, *, need_dw: bool = True, dx=None, dw=None, ws=None):
    """(dx, dw) of rmsnorm's y (gradient dy) and h (gradient dh or None); dx is the
    gradient of x and of the residual, dw is fp32 [d] (None unless need_dw)."""
    dev, dt, T, d = _rows(dy, "dy")
    _need(h, "h", dev, dt, (T, d))
    _need(w, "w", dev, dt, (d,))
    _need(rstd, "rstd", dev, _F32, (T,))
    if dh is not None:
        _need(dh, "dh", dev, dt, (T, d))
    dx = _out(dx, "dx", dev, dt, (T, d))
    if need_dw:
        dw = _out(dw, "dw", dev, _F32, (d,))
        if ws is None:
            ws = workspace(rmsnorm_backward_workspace_size(T, d), dev)
    _check(load().dora_rmsnorm_backward(_ptr(dy), _ptr(h), _ptr(w), _ptr(rstd), _ptr(dh), T, d, _DTYPE_CODE[dt],
                                        _ptr(dx), _ptr(dw) if need_dw else None, _ptr(ws), _nbytes(ws), _stream(dev)),
           "dora_rmsnorm_backward")
    return dx, (dw if need_dw else None)


# ------------------------------------------------------------ rows in 8 bits
def quantize_rows(x, col_scale=None, *, q=None, scale=None):
    """(q, scale): the rows of x * col_scale as int8 codes in [-127, 127] with an fp32 scale each."""
    dev, dt, n, d = _rows(x, "x")
    if col_scale is not None:
        _need(col_scale, "col_scale", dev, _F32, (d,))
    q = _out(q, "q", dev, _I8, (n, d))
    scale = _out(scale, "scale", dev, _F32, (n,))
    _check(load().dora_quantize_rows(_ptr(x), _ptr(col_scale), n, d, _DTYPE_CODE[dt], _ptr(q), _ptr(scale),
                                     _stream(dev)), "dora_quantize_rows")
    return q, scale


def dequantize_rows(q, scale, dtype: torch.dtype, *, out=None):
    """q * scale by rows, rounded once to dtype."""
    if not isinstance(q, torch.Tensor) or q.dim() != 2:
        raise ValueError("q must be a torch.Tensor of two dimensions")
    if dtype not in _DTYPE_CODE:
        raise ValueError(f"unsupported dtype {dtype}")
    dev = q.device
    n, d = q.shape
    _need(q, "q", dev, _I8)
    _need(scale, "scale", dev, _F32, (n,))
    out = _out(out, "out", dev, dtype, (n, d))
    _check(load().dora_dequantize_rows(_ptr(q), _ptr(scale), n, d, _DTYPE_CODE[dtype], _ptr(out), _stream(dev)),
           "dora_dequantize_rows")
    return out


# ------------------------------------------------------------ product
def matmul_q8(xq, xscale, wq, wscale=None, dtype: torch.dtype = torch.bfloat16, *, bias=None, g=None, lora_out=None,
              s: float = 1.0, out=None, ws=None):
    """y = base + ((g-1) base + (g s) lora_out) + bias, base = xscale wscale (xq wq^T) with the sum exact.

    xq int8 [T, d_in] with xscale fp32 [T], wq int8 [d_out, d_in] with wscale
    fp32 [d_out] (None: ones).  g fp32 [d_out] with lora_out [T, d_out] of
    dtype, and bias fp32 [d_out], are optional.  y has dtype.
    """
    for t, name in ((xq, "xq"), (wq, "wq")):
        if not isinstance(t, torch.Tensor) or t.dim() != 2:
            raise ValueError(f"{name} must be a torch.Tensor of two dimensions")
    if dtype not in _DTYPE_CODE:
        raise ValueError(f"unsupported dtype {dtype}")
    dev = xq.device
    T, K = xq.shape
    N = wq.shape[0]
    _need(xq, "xq", dev, _I8)
    _need(wq, "wq", dev, _I8, (N, K))
    _need(xscale, "xscale", dev, _F32, (T,))
    if wscale is not None:
        _need(wscale, "wscale", dev, _F32, (N,))
    if bias is not None:
        _need(bias, "bias", dev, _F32, (N,))
    if (g is None) != (lora_out is None):
        raise ValueError("g and lora_out are given together or not at all")
    if g is not None:
        _need(g, "g", dev, _F32, (N,))
        _need(lora_out, "lora_out", dev, dtype, (T, N))
    out = _out(out, "out", dev, dtype, (T, N))
    if ws is None:
        ws = workspace(matmul_q8_workspace_size(T, N, K), dev)
    _check(load().dora_matmul_q8(_ptr(xq), _ptr(xscale), _ptr(wq), _ptr(wscale), _ptr(bias), _ptr(g), _ptr(lora_out),
                                 float(s), T, N, K, _DTYPE_CODE[dtype], _ptr(out), _ptr(ws), _nbytes(ws),
                                 _stream(dev)), "dora_matmul_q8")
    return out


def linear_q8(x, wq, wscale, *, bias=None, g=None, lora_out=None, s: float = 1.0, out=None):
    """matmul_q8 of x [T, d_in], quantised by rows here; y has x's dtype."""
    xq, xscale = quantize_rows(x)
    return matmul_q8(xq, xscale, wq, wscale, x.dtype, bias=bias, g=g, lora_out=lora_out, s=s, out=out)


def linear_q8_backward(dy, wqt, wscale, *, out=None):
    """d_x of the linear map x -> x (wscale wq)^T, with dy * wscale quantised by rows.

    wqt int8 [d_in, d_out] is wq transposed, laid out once:
    wq.t().contiguous().
    """
    dq, dscale = quantize_rows(dy, wscale)
    return matmul_q8(dq, dscale, wqt, None, dy.dtype, out=out)


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
    def backward(ctx, dy):
        wqt, wscale = ctx.saved_tensors
        return linear_q8_backward(dy.contiguous(), wqt, wscale), None, None, None
