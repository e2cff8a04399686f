"""GPU parity of the 8-bit operators through the public entry points, against
the fp64 oracle on host copies of the very tensors the GPU path consumed.

Tolerances, derived from the arithmetic.  u = 2^-24 (fp32), U = the output
type's unit roundoff (2^-8 bf16, 2^-11 fp16, u fp32), and TINY the absolute
spacing of subnormals (2^-24 fp16; rounding then errs by half of it).
  h      one fp32 addition, one rounding: (U + u) |h|.
  rstd   the sum of squares is a chain of at most 64 terms per thread (or d/1024
         where rows are too long for registers) joined by 6 shuffles and 16
         waves: C = 90 + d/1024 additions of non-negative terms, relative error
         (C + 4) u with the squares' own; the root halves it; the division by
         d, the eps addition and the reciprocal root add 4 u.
  y      two products on top: (rstd's + 4 u + U) |y|.
  codes  q = rint(y / scale): y's two products and those in the row's largest,
         the scale's factor and product and the division round at most 8
         times, and rstd cancels: within 1/2 + 127 * 8 u of the exact quotient;
         scale: rstd's + 5 u.
  dx     c = sum u_j h_j errs by (C + 3) u sum|u h|; the rest is a few roundings
         of each term.
  dw     a chain of at most rows/parts + 7 + 64 additions: bounded by
         (T + 80) u sum|dy h rstd|.
  y of the product: the sum is exact; its conversion, two scales, the
         composition's terms and the bias round at most 8 times: 8 u times the
         sum of the terms' absolute values, and U |y|.
"""
import sys

import numpy as np
import pytest
import torch

import dora_adapter_factored_amd as D
from oracle import eightbit_oracle as O8
from parity_utils import host64

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
u = 2.0 ** -24
U = {"f32": u, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -24}
EPS = 1e-6


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def rng(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(g, *shape, dt=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dt)


def within(got, ref, bound, what):
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    bad = ~(np.abs(got - ref) <= bound)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(bad, np.abs(got - ref), -1)), bad.shape)
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} out of tolerance, worst at {i}: got {got[i]!r} "
                             f"ref {ref[i]!r} bound {np.broadcast_to(bound, bad.shape)[i]!r}")


def rstd_rel(d):
    return ((90 + d / 1024 + 4) / 2 + 4) * u


def check_codes(q, quot, what):
    q = host64(q)
    assert np.all(np.abs(q) <= 127), what
    within(q, quot, 0.5 + 127 * 8 * u, what)


def misaligned(t):
    buf = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
    v = buf[1:].view(t.shape)
    v.copy_(t)
    return v


# ------------------------------------------------------------------ norm
NORM_SHAPES = [
    # T, d: one token and many; one element; odd; each register form, and rows too long for them
    (1, 1), (1, 4096), (3, 7), (5, 64), (2, 65), (17, 1003), (9, 2056), (600, 512), (700, 1000), (520, 2048),
    (513, 4096), (515, 8200), (2, 28672), (3, 4099), (4, 33000), (513, 4101), (2, 65600),
]


@pytest.mark.parametrize("T,d", NORM_SHAPES)
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_rmsnorm(T, d, dt):
    say(f"[rmsnorm] {T}x{d} {dt}")
    g = rng(T * 31 + d)
    x, res = randn(g, T, d, dt=DT[dt]), randn(g, T, d, dt=DT[dt], scale=3.0)
    w = (1 + 0.2 * randn(g, d)).to(DT[dt])
    for r in (res, None):
        y, h, rstd = D.rmsnorm(x, w, EPS, r)
        q, scale, h2 = D.rmsnorm_q8(x, w, EPS, r)
        y3 = torch.empty_like(x)
        q3, scale3, _ = D.rmsnorm_q8(x, w, EPS, r, y=y3)
        torch.cuda.synchronize()
        assert torch.equal(h, h2) and torch.equal(q, q3) and torch.equal(scale, scale3) and torch.equal(y, y3)
        rh, rr, ry = O8.rmsnorm(host64(x), host64(w), EPS, None if r is None else host64(r))
        rel = rstd_rel(d)
        within(host64(h), rh, (U[dt] + u) * np.abs(rh) + TINY[dt], "h")
        within(host64(rstd), rr, rel * rr, "rstd")
        within(host64(y), ry, (rel + 4 * u + U[dt]) * np.abs(ry) + TINY[dt], "y")
        quot, rs = O8.to_codes(ry)
        check_codes(q, quot, "q")
        within(host64(scale), rs, (rel + 5 * u) * rs, "scale")


@pytest.mark.parametrize("T,d", [(1, 8192), (6, 1003), (600, 1024), (3, 70000)])
def test_rmsnorm_in_place(T, d):
    say(f"[rmsnorm] in place {T}x{d}")
    g = rng(d)
    x, res, w = randn(g, T, d, dt=torch.bfloat16), randn(g, T, d, dt=torch.bfloat16), randn(g, d, dt=torch.bfloat16)
    y, h, _ = D.rmsnorm(x, w, EPS, res)
    x1, r1 = x.clone(), res.clone()
    y1, h1, _ = D.rmsnorm(x1, w, EPS, res, h=x1)
    y2, h2, _ = D.rmsnorm(x, w, EPS, r1, h=r1)
    torch.cuda.synchronize()
    assert h1.data_ptr() == x1.data_ptr() and h2.data_ptr() == r1.data_ptr()
    assert torch.equal(h, x1) and torch.equal(h, r1) and torch.equal(y, y1) and torch.equal(y, y2)


def test_rmsnorm_misaligned_pointers():
    say("[rmsnorm] misaligned")
    g = rng(5)
    x, res, w = randn(g, 9, 512, dt=torch.bfloat16), randn(g, 9, 512, dt=torch.bfloat16), randn(g, 512, dt=torch.bfloat16)
    q, scale, h = D.rmsnorm_q8(x, w, EPS, res)
    # outputs and inputs a byte or an element off 16
    qb = torch.empty(9 * 512 + 1, dtype=torch.int8, device=DEV)[1:].view(9, 512)
    q1, s1, h1 = D.rmsnorm_q8(misaligned(x), misaligned(w), EPS, misaligned(res), q=qb, h=misaligned(h))
    torch.cuda.synchronize()
    assert torch.equal(h, h1)
    assert torch.equal(q, q1) and torch.equal(scale, s1)   # the same sums in the same order


@pytest.mark.parametrize("d", [1024, 1003, 70000])
def test_rows_of_zeros_nan_and_infinity(d):
    say(f"[8 bits] special rows, d={d}")
    g = rng(7)
    x = randn(g, 6, d)
    x[0] = 0.0
    x[1, d // 2] = float("nan")
    x[2, d - 1] = float("inf")
    x[3, 0] = float("-inf")
    x[4] = 2.0 ** -130
    w = torch.ones(d, device=DEV)
    for q, scale in (D.quantize_rows(x), D.rmsnorm_q8(x, w, EPS)[:2]):
        v = D.dequantize_rows(q, scale, torch.float32)
        torch.cuda.synchronize()
        assert torch.all(q[:5] == 0) and torch.all(scale[[0, 4]] == 0) and torch.all(torch.isnan(scale[1:4]))
        assert torch.all(v[[0, 4]] == 0) and torch.all(torch.isnan(v[1:4])) and torch.all(torch.isfinite(v[5]))
        assert int(q[5].abs().max()) == 127
    # and the rows of a product that they reach, no others
    wq, ws = D.quantize_rows(randn(g, 40, d))
    xq, xs = D.quantize_rows(x)
    y = D.matmul_q8(xq, xs, wq, ws, torch.float32)
    torch.cuda.synchronize()
    assert torch.all(torch.isnan(y[1:4])) and torch.all(torch.isfinite(y[[0, 4, 5]])) and torch.all(y[[0, 4]] == 0)


def test_empty_calls():
    x = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(64, dtype=torch.bfloat16, device=DEV)
    y, h, rstd = D.rmsnorm(x, w, EPS, x)
    dx, dw = D.rmsnorm_backward(x, x, w, rstd)
    q, scale = D.quantize_rows(x)
    wq, ws = D.quantize_rows(torch.ones(8, 64, device=DEV))
    out = D.matmul_q8(q, scale, wq, ws)
    torch.cuda.synchronize()
    assert y.shape == (0, 64) and dx.shape == (0, 64) and torch.all(dw == 0) and out.shape == (0, 8)


BWD_SHAPES = [(1, 1), (1, 4096), (3, 7), (17, 1003), (300, 65), (600, 512), (1100, 2048), (515, 8200), (2, 28672),
              (3, 4099), (530, 4201), (520, 9001), (3, 30721), (3, 66000)]


@pytest.mark.parametrize("T,d", BWD_SHAPES)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_rmsnorm_backward(T, d, dt):
    say(f"[rmsnorm backward] {T}x{d} {dt}")
    g = rng(T + d)
    dy, h, dh = (randn(g, T, d, dt=DT[dt]) for _ in range(3))
    w = (1 + 0.2 * randn(g, d)).to(DT[dt])
    rstd = torch.rsqrt(h.float().square().mean(1) + EPS)
    C = 90 + d / 1024
    H, R, DY, W = host64(h), host64(rstd), host64(dy), host64(w)
    uh = np.mean(np.abs(DY * W * H), axis=1, keepdims=True)
    for extra in (dh, None):
        dx, dw = D.rmsnorm_backward(dy, h, w, rstd, extra)
        dx2, none = D.rmsnorm_backward(dy, h, w, rstd, extra, need_dw=False)
        dx3, dw3 = D.rmsnorm_backward(dy, h, w, rstd, extra)
        torch.cuda.synchronize()
        assert none is None and torch.equal(dx, dx2) and torch.equal(dx, dx3) and torch.equal(dw, dw3)
        rdx, rdw = O8.rmsnorm_backward(DY, H, W, R, None if extra is None else host64(extra))
        r = R[:, None]
        size = np.abs(r * DY * W) + np.abs(H) * r ** 3 * uh + (0 if extra is None else np.abs(host64(extra)))
        bound = np.abs(H) * r ** 3 * (C + 3) * u * uh + 8 * u * size + U[dt] * np.abs(rdx) + TINY[dt]
        within(host64(dx), rdx, bound, "dx")
        within(host64(dw), rdw, (T + 80) * u * np.sum(np.abs(DY * H * r), axis=0), "dw")
    inplace = dy.clone()
    dx4, _ = D.rmsnorm_backward(inplace, h, w, rstd, None, dx=inplace)
    torch.cuda.synchronize()
    assert torch.equal(inplace, dx)


def test_rmsnorm_gradient_against_differences():
    # central differences of the fp64 definition along random directions: the
    # loss is cubic-smooth in a step of 1e-4, so the difference errs by about
    # 1e-8 and 1e-11 (rounding); the fp32 gradient by some 1e-5 of its size
    say("[rmsnorm] gradient against differences")
    g = rng(11)
    T, d = 6, 130
    x, res = randn(g, T, d).requires_grad_(), randn(g, T, d).requires_grad_()
    w = (1 + 0.2 * randn(g, d)).requires_grad_()
    cy, ch = randn(g, T, d), randn(g, T, d)
    y, h = D.RMSNorm.apply(x, res, w, EPS)
    (y * cy + h * ch).sum().backward()
    torch.cuda.synchronize()
    X, S, W, CY, CH = (host64(t) for t in (x, res, w, cy, ch))

    def loss(a, b, c):
        hh, _, yy = O8.rmsnorm(a, c, EPS, b)
        return np.sum(yy * CY + hh * CH)

    r = np.random.default_rng(3)
    for which, grad in ((0, x.grad), (1, res.grad), (2, w.grad)):
        for _ in range(4):
            args = [X, S, W]
            v = r.standard_normal(args[which].shape)
            step = [a + (1e-4 * v if i == which else 0) for i, a in enumerate(args)]
            back = [a - (1e-4 * v if i == which else 0) for i, a in enumerate(args)]
            diff = (loss(*step) - loss(*back)) / 2e-4
            got = np.sum(host64(grad) * v)
            assert abs(got - diff) <= 1e-5 * np.sum(np.abs(host64(grad) * v)) + 1e-6, (which, got, diff)


def test_rmsnorm_autograd_paths():
    say("[rmsnorm] autograd: no residual, frozen w, unused h")
    g = rng(12)
    x = randn(g, 5, 96, dt=torch.bfloat16).requires_grad_()
    w = randn(g, 96, dt=torch.bfloat16)
    dy = randn(g, 5, 96, dt=torch.bfloat16)
    y = D.RMSNorm.apply(x, None, w, EPS)
    y.backward(dy)
    _, h, rstd = D.rmsnorm(x.detach(), w, EPS)
    dx, _ = D.rmsnorm_backward(dy, h, w, rstd)
    assert torch.equal(x.grad, dx)
    res = randn(g, 5, 96, dt=torch.bfloat16).requires_grad_()
    x.grad = None
    y, h = D.RMSNorm.apply(x, res, w, EPS)
    y.backward(dy)
    _, h2, rstd = D.rmsnorm(x.detach(), w, EPS, res.detach())
    dx, _ = D.rmsnorm_backward(dy, h2, w, rstd)
    assert torch.equal(x.grad, dx) and torch.equal(res.grad, dx)
    x.grad = res.grad = None
    y, h = D.RMSNorm.apply(x, res, w, EPS)
    h.backward(dy)
    assert torch.equal(x.grad, dy) and torch.equal(res.grad, dy)


# ------------------------------------------------------------------ rows in 8 bits
@pytest.mark.parametrize("n,d", [(1, 1), (1, 27648), (7, 1003), (4, 64), (600, 2056), (520, 5120), (3, 70000)])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_quantize_rows(n, d, dt):
    say(f"[quantize] {n}x{d} {dt}")
    g = rng(n + d)
    x = randn(g, n, d, dt=DT[dt], scale=2.0)
    cs = randn(g, d).abs() + 0.1
    for c in (None, cs):
        q, scale = D.quantize_rows(x, c)
        v = D.dequantize_rows(q, scale, DT[dt])
        torch.cuda.synchronize()
        p = host64(x) if c is None else host64(x) * host64(c)
        quot, rs = O8.to_codes(p)
        check_codes(q, quot, "q")
        within(host64(scale), rs, 5 * u * rs, "scale")
        ref = host64(q) * host64(scale)[:, None]
        within(host64(v), ref, (U[dt] + u) * np.abs(ref) + TINY[dt], "values")


def test_quantize_ties_go_to_even():
    # scale = 127/127 = 1: the codes are the rounded values themselves
    x = torch.tensor([[127.0, 0.5, 1.5, 2.5, -0.5, -1.5, -2.5, 126.5]], device=DEV)
    q, scale = D.quantize_rows(x)
    torch.cuda.synchronize()
    assert q.tolist() == [[127, 0, 2, 2, 0, -2, -2, 126]] and scale.tolist() == [1.0]


# ------------------------------------------------------------------ product
def check_product(T, N, K, dt, adapter=False, bias=False, scaled=True, seed=0, reference=True):
    g = rng(seed + T * 7 + N * 3 + K)
    xq = torch.randint(-127, 128, (T, K), generator=g, device=DEV, dtype=torch.int8)
    wq = torch.randint(-127, 128, (N, K), generator=g, device=DEV, dtype=torch.int8)
    xs = torch.rand(T, generator=g, device=DEV) * 0.01 + 1e-3
    ws = torch.rand(N, generator=g, device=DEV) * 0.01 + 1e-3 if scaled else None
    if not scaled:
        xs = xs * 1e-2   # keeps the results inside fp16
    gg = 1 + 0.3 * randn(g, N) if adapter else None
    lora = randn(g, T, N, dt=DT[dt]) if adapter else None
    b = randn(g, N) if bias else None
    s = 1.7 if adapter else 1.0
    y = D.matmul_q8(xq, xs, wq, ws, DT[dt], bias=b, g=gg, lora_out=lora, s=s)
    torch.cuda.synchronize()
    if not reference:
        return y, (xq, xs, wq, ws, gg, lora, b, s)
    h = lambda t: None if t is None else host64(t)  # noqa: E731
    s32 = float(np.float32(s))
    ref, size = O8.matmul_q8(xq.cpu().numpy(), h(xs), wq.cpu().numpy(), h(ws), h(b), h(gg), h(lora), s32)
    within(host64(y), ref, 8 * u * size + U[dt] * np.abs(ref) + TINY[dt], f"y {T}x{N}x{K}")
    return y, (xq, xs, wq, ws, gg, lora, b, s)


PRODUCT_SIZES = [
    (1, 1, 1), (1, 16, 128), (1, 17, 129), (2, 4096, 4096), (1, 1024, 5120), (3, 130, 2056), (4, 48, 127), (5, 33, 1003),
    (8, 512, 8192), (15, 100, 64), (16, 256, 1024), (17, 4090, 2056), (31, 200, 1024), (33, 65, 255), (48, 512, 4096),
    (64, 512, 512), (65, 300, 640), (100, 129, 1003), (128, 128, 128), (128, 1024, 4096), (130, 257, 2056),
    (200, 1000, 48), (256, 256, 256), (257, 511, 1040), (333, 4090, 2056), (512, 768, 1001), (300, 5120, 1024),
    (1000, 520, 16), (700, 1, 300), (2048, 64, 520), (513, 2050, 8200),
]


@pytest.mark.parametrize("T,N,K", PRODUCT_SIZES)
def test_matmul_q8_sizes(T, N, K):
    say(f"[matmul_q8] {T}x{N}x{K}")
    check_product(T, N, K, "bf16")
    check_product(T, N, K, "f32", adapter=True, bias=True)


# sizes whose least cost each of the tile forms has, alone and in parts of K
# (the reference sums on the GPU in fp64, where every sum is exact)
FORM_SIZES = [
    # 256 x 256, 192 x 256, 128 x 256, 128 x 128, 64 x 128, 64 x 64 in one part
    (1814, 6529, 36), (2048, 8192, 384), (900, 8847, 36), (1030, 8200, 264), (523, 7234, 100), (520, 8200, 264),
    (1753, 1225, 36), (300, 7000, 2000), (65, 8740, 40), (200, 512, 1028), (74, 631, 68),
    # and in parts
    (441, 5414, 8276), (134, 5554, 6244), (260, 3780, 5092), (70, 3273, 5676), (513, 2050, 8200), (75, 2113, 4332),
    (65, 884, 2064), (48, 512, 4100),
    # rows that are not 4-byte aligned: through registers, or padded first
    (200, 900, 2049), (100, 129, 131), (2000, 1300, 1301), (1900, 2051, 130),
]


@pytest.mark.parametrize("T,N,K", FORM_SIZES)
def test_matmul_q8_forms(T, N, K):
    say(f"[matmul_q8 forms] {T}x{N}x{K}")
    for dt, adapter, bias in (("bf16", False, True), ("f32", True, False)):
        y, (xq, xs, wq, ws, g, lora, b, s) = check_product(T, N, K, dt, adapter, bias, reference=False)
        base = ((xq.double() @ wq.double().t()) * xs.double()[:, None]) * ws.double()
        ref, size = base.clone(), base.abs()
        if adapter:
            extra = (g.double() * float(np.float32(s))) * lora.double()
            ref = ref + (g.double() - 1) * base + extra
            size = size + ((g.double() - 1) * base).abs() + extra.abs()
        if bias:
            ref, size = ref + b.double(), size + b.double().abs()
        bad = (y.double() - ref).abs() > 8 * u * size + U[dt] * ref.abs() + TINY[dt]
        assert not bool(bad.any()), (T, N, K, dt, int(bad.sum()), bad.nonzero()[:4].tolist())


@pytest.mark.parametrize("T,N,K", [(1, 300, 1024), (24, 300, 1024), (24, 301, 1001), (150, 300, 1024), (300, 301, 1001),
                                   (600, 1024, 2048)])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("adapter,bias,scaled", [(True, False, True), (False, True, True), (False, False, False),
                                                 (True, True, False)])
def test_matmul_q8_epilogues(T, N, K, dt, adapter, bias, scaled):
    say(f"[matmul_q8] {T}x{N}x{K} {dt} adapter={adapter} bias={bias} wscale={scaled}")
    check_product(T, N, K, dt, adapter, bias, scaled)


@pytest.mark.parametrize("T", [1, 20, 150, 300])
def test_matmul_q8_longest_sums_stay_in_int32(T):
    say(f"[matmul_q8] longest sums, T={T}")
    K = 131071
    xq = torch.full((T, K), -128, dtype=torch.int8, device=DEV)
    wq = torch.full((34, K), -128, dtype=torch.int8, device=DEV)
    wq[1::2] = 127
    one = torch.ones(T, device=DEV)
    y = D.matmul_q8(xq, one, wq, None, torch.float32)
    torch.cuda.synchronize()
    assert torch.all(y[:, 0::2] == float(np.float32(K * 16384))) and torch.all(y[:, 1::2] == float(np.float32(-K * 16256)))


@pytest.mark.parametrize("N,K", [(512, 2048), (301, 1003), (5120, 5120)])
def test_matmul_q8_rows_do_not_depend_on_the_batch(N, K):
    # the sum is exact and the rest is the same arithmetic for every form of
    # the kernel, so a token's result is bitwise the same in any batch
    say(f"[matmul_q8] batches, {N}x{K}")
    y, (xq, xs, wq, ws, g, lora, b, s) = check_product(700, N, K, "bf16", adapter=True, bias=True)
    for lo, hi in ((0, 1), (3, 7), (10, 40), (100, 170), (200, 500)):
        part = D.matmul_q8(xq[lo:hi].contiguous(), xs[lo:hi].contiguous(), wq, ws, torch.bfloat16, bias=b, g=g,
                           lora_out=lora[lo:hi].contiguous(), s=s)
        torch.cuda.synchronize()
        assert torch.equal(part, y[lo:hi]), (lo, hi)


def test_matmul_q8_misaligned_codes_and_in_place():
    say("[matmul_q8] misaligned codes; y over lora_out")
    # the last one through registers in 128 x 128 tiles
    for T, N, K in ((1, 260, 1024), (2, 260, 1024), (40, 260, 1024), (300, 260, 1024), (2000, 1300, 1300)):
        y, (xq, xs, wq, ws, g, lora, b, s) = check_product(T, N, K, "bf16", adapter=True)
        mis = D.matmul_q8(misaligned(xq), xs, misaligned(wq), ws, torch.bfloat16, g=g, lora_out=misaligned(lora), s=s,
                          out=misaligned(y))
        over = lora.clone()
        D.matmul_q8(xq, xs, wq, ws, torch.bfloat16, g=g, lora_out=over, s=s, out=over)
        torch.cuda.synchronize()
        assert torch.equal(mis, y) and torch.equal(over, y)


@pytest.mark.parametrize("T", [1, 40, 300])
def test_matmul_q8_on_a_side_stream_and_captured(T):
    say(f"[matmul_q8] side stream, graph, T={T}")
    y, (xq, xs, wq, ws, *_r) = check_product(T, 1024, 2048, "bf16")
    x = torch.randn(T, 2048, device=DEV, dtype=torch.bfloat16, generator=rng(1))
    want = D.linear_q8(x, wq, ws)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = D.matmul_q8(xq, xs, wq, ws)
        lin = D.linear_q8(x, wq, ws)
    side.synchronize()
    assert torch.equal(got, y) and torch.equal(lin, want)
    graph = torch.cuda.CUDAGraph()
    out = torch.empty_like(want)
    with torch.cuda.graph(graph):
        D.linear_q8(x, wq, ws, out=out)
    for k in range(3):
        x2 = torch.randn(T, 2048, device=DEV, dtype=torch.bfloat16, generator=rng(20 + k))
        eager = D.linear_q8(x2, wq, ws)
        x.copy_(x2)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager), k


def test_matmul_q8_offsets_past_32_bits():
    # y and lora_out of more than 2^31 elements' bytes: the last rows against
    # the same rows alone
    say("[matmul_q8] large offsets")
    T, N, K = 36000, 70000, 32
    g = rng(9)
    xq = torch.randint(-127, 128, (T, K), generator=g, device=DEV, dtype=torch.int8)
    wq = torch.randint(-127, 128, (N, K), generator=g, device=DEV, dtype=torch.int8)
    xs, ws = torch.rand(T, generator=g, device=DEV), torch.rand(N, generator=g, device=DEV)
    y = D.matmul_q8(xq, xs, wq, ws)
    tail = D.matmul_q8(xq[-70:].contiguous(), xs[-70:].contiguous(), wq, ws)
    torch.cuda.synchronize()
    assert y.numel() > 2 ** 31 and torch.equal(y[-70:], tail)


@pytest.mark.parametrize("N,K", [(40, 64), (17, 9)])
def test_matmul_q8_more_tokens_than_one_launch_takes(N, K):
    say(f"[matmul_q8] many tokens, {N}x{K}")
    T = (1 << 19) + 70
    g = rng(N)
    xq = torch.randint(-127, 128, (T, K), generator=g, device=DEV, dtype=torch.int8)
    wq = torch.randint(-127, 128, (N, K), generator=g, device=DEV, dtype=torch.int8)
    xs, ws = torch.rand(T, generator=g, device=DEV), torch.rand(N, generator=g, device=DEV)
    gg, lora = torch.rand(N, generator=g, device=DEV), randn(g, T, N)
    y = D.matmul_q8(xq, xs, wq, ws, torch.float32, g=gg, lora_out=lora, s=0.5)
    base = (xq.double() @ wq.double().t()) * xs.double()[:, None] * ws.double()
    extra = (gg.double() * 0.5) * lora.double()
    bad = (y.double() - (gg.double() * base + extra)).abs() > 9 * u * (3 * base.abs() + extra.abs()) + TINY["f32"]
    assert not bool(bad.any())


# ------------------------------------------------------------------ a training step's frozen weight
@pytest.mark.parametrize("T,N,K", [(1, 64, 96), (70, 130, 200), (300, 512, 384)])
def test_linear_q8_and_its_gradient(T, N, K):
    """y and d_x against the formulas in 64 bits on the codes that the GPU made,
    and d_x against the gradient of the linear map itself: quantising p = dy ws
    errs by at most half a step per element, so |d_x - exact| <= step/2 sum_n
    |wq_nk| (and the roundings).  The map is linear: its gradient along v is its
    difference, (f(x + v) - f(x)) . dy, whatever the step."""
    say(f"[linear_q8] {T}x{N}x{K}")
    g = rng(T)
    wq, ws = D.quantize_rows(randn(g, N, K, scale=K ** -0.5))
    wqt = wq.t().contiguous()
    x = randn(g, T, K).requires_grad_()
    dy = randn(g, T, N)
    y = D.LinearQ8.apply(x, wq, ws, wqt)
    y.backward(dy)
    xq, xs = D.quantize_rows(x.detach())
    dq, ds = D.quantize_rows(dy, ws)
    torch.cuda.synchronize()
    ref, size = O8.matmul_q8(xq.cpu().numpy(), host64(xs), wq.cpu().numpy(), host64(ws))
    within(host64(y.detach()), ref, 8 * u * size + u * np.abs(ref), "y")
    ref, size = O8.matmul_q8(dq.cpu().numpy(), host64(ds), wqt.cpu().numpy())
    within(host64(x.grad), ref, 8 * u * size + u * np.abs(ref), "dx")
    Wd = host64(wq) * host64(ws)[:, None]
    exact = host64(dy) @ Wd
    step = host64(ds)[:, None] * np.abs(host64(wq)).sum(axis=0)
    within(host64(x.grad), exact, step * (0.5 + 1e-3) + 1e-5 * np.abs(exact), "dx against the linear map")
    v = np.random.default_rng(1).standard_normal((T, K))
    X = host64(x.detach())
    diff = np.sum(((X + v) @ Wd.T - X @ Wd.T) * host64(dy))
    assert abs(np.sum(host64(x.grad) * v) - diff) <= np.sum(np.abs(v) * (step * (0.5 + 1e-3) + 1e-5 * np.abs(exact)))


def test_example_block():
    """The example's block at small sizes.  Each 8-bit rounding errs by at most
    half a step of 1/127 of its row's largest value, some 1% of a normal row's
    rms; four of them (two weights, two activations) add to under 2% in the
    2-norm, bf16 roundings to under 1% more."""
    say("[example] 8-bit block")
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "eight_bit_block.py")
    spec = importlib.util.spec_from_file_location("eight_bit_block", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    off, loss, grads = mod.main(["--hidden", "512", "--inner", "1024", "--rank", "8", "--tokens", "70"])
    assert all(v < 0.03 for v in off.values()), off
    assert bool(torch.isfinite(loss)) and all(bool(torch.isfinite(g).all()) and float(g.float().norm()) > 0 for g in grads.values())
