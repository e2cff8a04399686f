"""The row operators and the frozen layer's gradient where the other tests do not
reach: fp16, pointers off 16 bytes with rows that are whole packs, dx written
over dh, rows that hold a NaN or an infinity.

Bounds are those of test_eightbit.py: dx errs by (C + 3) u of its reduction's
terms and 8 u of its own, dw by (T + 80) u of its terms, each rounded once to its
type.  Where the arithmetic is the same in the same order, results are equal.
"""
import sys

import numpy as np
import pytest
import torch

import dora_adapter_factored_amd as D
from oracle import eightbit_oracle as O8
from parity_utils import host64
from test_eightbit import BWD_SHAPES, DEV, DT, EPS, TINY, U, misaligned, randn, rng, u, within

pytestmark = pytest.mark.gpu


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def backward_inputs(T, d, dt):
    g = rng(T + d)
    dy, h, dh = (randn(g, T, d, dt=DT[dt]) for _ in range(3))
    w = (1 + 0.2 * randn(g, d)).to(DT[dt])
    return dy, h, dh, w, torch.rsqrt(h.float().square().mean(1) + EPS)


@pytest.mark.parametrize("T,d", BWD_SHAPES + [(520, 16384), (40, 30720), (700, 2048)])
def test_rmsnorm_backward_f16(T, d):
    say(f"[rmsnorm backward] {T}x{d} f16")
    dy, h, dh, w, rstd = backward_inputs(T, d, "f16")
    C = 90 + d / 1024
    H, R, DY, W = host64(h), host64(rstd), host64(dy), host64(w)
    uh = np.mean(np.abs(DY * W * H), axis=1, keepdims=True)
    for extra in (dh, None):
        dx, dw = D.rmsnorm_backward(dy, h, w, rstd, extra)
        torch.cuda.synchronize()
        rdx, rdw = O8.rmsnorm_backward(DY, H, W, R, None if extra is None else host64(extra))
        r = R[:, None]
        size = np.abs(r * DY * W) + np.abs(H) * r ** 3 * uh + (0 if extra is None else np.abs(host64(extra)))
        bound = np.abs(H) * r ** 3 * (C + 3) * u * uh + 8 * u * size + U["f16"] * np.abs(rdx) + TINY["f16"]
        within(host64(dx), rdx, bound, "dx")
        within(host64(dw), rdw, (T + 80) * u * np.sum(np.abs(DY * H * r), axis=0), "dw")


# register forms of one, two, four and the most packs a thread, and rows too long for them
ROWS = [(9, 512), (600, 2048), (600, 8192), (520, 9216), (3, 28672), (3, 70000)]


@pytest.mark.parametrize("T,d", ROWS)
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_backward_misaligned_and_in_place(T, d, dt):
    say(f"[rmsnorm backward] misaligned, in place {T}x{d} {dt}")
    dy, h, dh, w, rstd = backward_inputs(T, d, dt)
    dx, dw = D.rmsnorm_backward(dy, h, w, rstd, dh)
    out = misaligned(dx)
    dx1, dw1 = D.rmsnorm_backward(misaligned(dy), misaligned(h), misaligned(w), rstd, misaligned(dh), dx=out)
    over_dh, over_dy = dh.clone(), dy.clone()
    D.rmsnorm_backward(dy, h, w, rstd, over_dh, dx=over_dh)
    D.rmsnorm_backward(over_dy, h, w, rstd, dh, dx=over_dy)
    torch.cuda.synchronize()
    assert dx1.data_ptr() == out.data_ptr() and dx1.data_ptr() % 16 != 0
    assert torch.equal(dx, dx1) and torch.equal(dw, dw1)
    assert torch.equal(dx, over_dh) and torch.equal(dx, over_dy)


@pytest.mark.parametrize("n,d", ROWS + [(1, 16), (700, 5120)])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_rows_to_8_bits_and_back_misaligned(n, d, dt):
    say(f"[8 bits] misaligned {n}x{d} {dt}")
    g = rng(n + d)
    x, cs = randn(g, n, d, dt=DT[dt]), torch.rand(d, generator=g, device=DEV) + 0.5
    for c in (None, cs):
        q, scale = D.quantize_rows(x, c)
        v = D.dequantize_rows(q, scale, DT[dt])
        qb = torch.empty(n * d + 1, dtype=torch.int8, device=DEV)[1:].view(n, d)
        q1, s1 = D.quantize_rows(misaligned(x), None if c is None else misaligned(c), q=qb)
        v1 = D.dequantize_rows(q1, s1, DT[dt], out=misaligned(v))
        torch.cuda.synchronize()
        assert torch.equal(q, q1) and torch.equal(scale, s1) and torch.equal(v, v1)


@pytest.mark.parametrize("d", [1024, 1003, 9216, 28672, 70000])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_backward_rows_of_nan_and_infinity(d, dt):
    """A NaN or an infinity in a row's dy or h makes that row of dx NaN through
    its mean, and the columns of dw that it stands in; a NaN in dh its own
    element.  The other rows and columns are what they are without it."""
    say(f"[rmsnorm backward] special rows, d={d} {dt}")
    T, j, k = 7, d // 2, d - 1
    dy, h, dh, w, rstd = backward_inputs(T, d, dt)
    dx0, dw0 = D.rmsnorm_backward(dy, h, w, rstd, dh)
    nan, inf = float("nan"), float("inf")
    dy[1, j] = nan
    dy[2, j] = inf
    h[3, k] = nan
    h[4, k] = -inf
    dh[5, 0] = nan
    rstd[4] = 0.0   # as the forward pass keeps it for a row with an infinity
    dx, dw = D.rmsnorm_backward(dy, h, w, rstd, dh)
    torch.cuda.synchronize()
    assert bool(torch.isnan(dx[[1, 3, 4]]).all())
    assert not bool(torch.isfinite(dx[2]).any())   # an infinite mean times h, or NaN
    assert torch.equal(dx[[0, 6]], dx0[[0, 6]]) and torch.equal(dx[5, 1:], dx0[5, 1:]) and bool(torch.isnan(dx[5, 0]))
    bad = torch.zeros(d, dtype=torch.bool, device=DEV)
    bad[[j, k]] = True
    assert bool(torch.isnan(dw[k])) and not bool(torch.isfinite(dw[j])) and bool(torch.isfinite(dw[~bad]).all())


@pytest.mark.parametrize("T,N,K", [(1, 64, 96), (70, 130, 200), (300, 512, 384)])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_linear_q8_gradient_in_16_bits(T, N, K, dt):
    """d_x against the codes that the GPU made (8 u of the terms, one rounding),
    and against the gradient of the linear map: half a step of each rounded
    element of dy ws, and the same rounding."""
    say(f"[linear_q8] {T}x{N}x{K} {dt}")
    g = rng(T)
    wq, ws = D.quantize_rows(randn(g, N, K, scale=K ** -0.5))
    wqt = wq.t().contiguous()
    x = randn(g, T, K, dt=DT[dt]).requires_grad_()
    dy = randn(g, T, N, dt=DT[dt])
    y = D.LinearQ8.apply(x, wq, ws, wqt)
    y.backward(dy)
    xq, xs = D.quantize_rows(x.detach())
    dq, ds = D.quantize_rows(dy, ws)
    torch.cuda.synchronize()
    assert y.dtype == DT[dt] and x.grad.dtype == DT[dt]
    ref, size = O8.matmul_q8(xq.cpu().numpy(), host64(xs), wq.cpu().numpy(), host64(ws))
    within(host64(y.detach()), ref, 8 * u * size + U[dt] * np.abs(ref) + TINY[dt], "y")
    ref, size = O8.matmul_q8(dq.cpu().numpy(), host64(ds), wqt.cpu().numpy())
    within(host64(x.grad), ref, 8 * u * size + U[dt] * np.abs(ref) + TINY[dt], "dx")
    exact = host64(dy) @ (host64(wq) * host64(ws)[:, None])
    step = host64(ds)[:, None] * np.abs(host64(wq)).sum(axis=0)
    within(host64(x.grad), exact, (step * (0.5 + 1e-3) + 1e-5 * np.abs(exact)) * (1 + U[dt]) + U[dt] * np.abs(exact) + TINY[dt],
           "dx against the linear map")
