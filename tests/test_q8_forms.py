"""Each form of the 8-bit product, alone and in parts of K, at sizes for which
csrc/dora_q8_plan.h chooses it: the choice on the host (the header built by the
host compiler), the results on the GPU.

The tolerance is that of the product's other tests: the sum is exact, its
conversion, two scales, the composition's terms and the bias round at most 8
times (8 u times the sum of the terms' absolute values, u = 2^-24), and the
result once more to its type.  The reference sums in fp64 on the GPU, where
every sum of codes' products is exact.
"""
import os
import shutil
import subprocess
import sys

import pytest
import torch

import dora_adapter_factored_amd as D

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "dora_adapter_factored_amd", "csrc")

CHECKER = r"""
#include <cstdio>
#include <cstdlib>
#include "dora_q8_plan.h"
using namespace dora;
int main(int argc, char** argv) {   // T N K aligned ... -> form, parts, form and parts of the padded product, bytes
    for (int i = 1; i + 3 < argc; i += 4) {
        const int64_t T = atoll(argv[i]), N = atoll(argv[i + 1]), K = atoll(argv[i + 2]);
        const Q8Plan p = plan_q8(T, N, K, atoi(argv[i + 3]) != 0);
        const Q8Plan in = p.form == kPadded ? plan_pad(T, N, K).plan : Q8Plan{0, 0};
        printf("%d %d %d %d %zu\n", p.form, p.ks, in.form, in.ks, q8_workspace_bytes(T, N, K));
    }
}
"""
DIRECT, ONE_TOKEN, PADDED, REGS_BIG, REGS_SMALL = -1, -2, -3, 6, 7

# T, d_out, d_in: the form, whether it takes parts of K, the padded product's
# form.  Forms 0 to 5: tiles of 256 x 256, 192 x 256, 128 x 256, 128 x 128, 64 x
# 128 and 64 x 64.
FORMS = [
    ((2146, 5542, 256), 0, False, None), ((400, 5572, 8212), 0, True, None),
    ((1565, 4913, 260), 1, False, None), ((131, 5610, 5892), 1, True, None),
    ((1670, 2317, 256), 2, False, None), ((2788, 130, 12236), 2, True, None),
    ((322, 5525, 268), 3, False, None), ((66, 3310, 5204), 3, True, None),
    ((131, 5490, 256), 4, False, None), ((2, 4108, 10920), 4, True, None),
    ((17, 64, 256), 5, False, None), ((2, 64, 12716), 5, True, None),
    ((1, 4090, 2056), ONE_TOKEN, False, None), ((1, 301, 1001), ONE_TOKEN, False, None),
    ((12, 1024, 5120), DIRECT, False, None), ((2, 65, 257), DIRECT, False, None), ((300, 70, 15), DIRECT, False, None),
    ((322, 5525, 270), REGS_BIG, False, None), ((200, 64, 274), REGS_SMALL, False, None),
    ((2146, 5542, 257), PADDED, False, 0), ((400, 5572, 8213), PADDED, True, 0),
    ((2056, 3849, 257), PADDED, False, 1), ((133, 5453, 6265), PADDED, True, 1),
    ((2435, 2053, 387), PADDED, False, 2), ((2358, 138, 14062), PADDED, True, 2),
    ((1669, 1157, 1154), PADDED, False, 3), ((65, 2691, 8623), PADDED, True, 3),
    ((772, 1234, 1794), PADDED, False, 4), ((1647, 65, 5721), PADDED, True, 4),
    ((1799, 1040, 3469), PADDED, False, 5), ((70, 791, 7333), PADDED, True, 5),
]


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    d = tmp_path_factory.mktemp("q8plan")
    (d / "check.cpp").write_text(CHECKER)
    subprocess.run([cxx, "-std=c++17", "-O1", "-I", CSRC, str(d / "check.cpp"), "-o", str(d / "check")], check=True)

    def run(T, N, K, aligned):
        out = subprocess.run([str(d / "check"), str(T), str(N), str(K), str(int(aligned))], check=True, capture_output=True,
                             text=True).stdout.split()
        return tuple(int(x) for x in out)

    return run


@pytest.mark.parametrize("size,form,parts,inner", FORMS)
def test_sizes_take_their_forms(plan, size, form, parts, inner):
    got, ks, got_inner, inner_ks, nbytes = plan(*size, size[2] % 4 == 0)
    assert got == form
    if form == PADDED:
        assert got_inner == inner and (inner_ks > 1) == parts
    else:
        assert (ks > 1) == parts
    assert nbytes == D.matmul_q8_workspace_size(*size)


# d_in that is no multiple of 4: measured GPU times in us on MI355X with weights
# that are not in the last-level cache, of the form straight from memory (up to
# 64 tokens), the padded product, and 64 x 64 and 128 x 128 tiles through registers
ODD = [
    ((24, 5120, 27649), 149.2, 80.1, 98.1, 209.9), ((64, 5120, 27649), 265.4, 89.6, 135.7, 251.3),
    ((16, 5120, 27649), 107.4, 81.0, 92.7, 203.1), ((2, 5120, 27649), 69.0, 80.0, 86.3, 195.0),
    ((64, 300, 1001), 4.3, 9.2, 8.8, 15.5), ((64, 1299, 1001), 6.1, 10.2, 9.2, 16.3), ((64, 777, 2050), 6.0, 12.3, 11.5, 22.5),
    ((48, 4096, 14339), 74.9, 40.3, 64.8, 126.3), ((16, 12001, 4097), 27.4, 35.8, 21.9, 38.2),
    ((24, 1025, 5121), 10.5, 17.8, 20.1, 42.6), ((64, 4099, 4099), 30.3, 21.3, 18.7, 36.2), ((64, 8193, 8193), 112.9, 45.0, 44.7, 80.9),
    ((100, 8193, 8193), None, 51.0, 61.9, 90.4), ((333, 8193, 8193), None, 71.0, 116.1, 85.8),
    ((100, 28673, 2049), None, 46.2, 46.2, 34.4), ((1000, 515, 16385), None, 34.9, 53.8, 128.3),
    ((1000, 4099, 4099), None, 52.3, 70.5, 82.7), ((2000, 4099, 4099), None, 68.1, 128.4, 121.0),
    ((2000, 12001, 4097), None, 165.1, 350.9, 264.6),
]


@pytest.mark.parametrize("size,direct,padded,small,big", ODD)
def test_rows_of_odd_length_take_a_form_that_is_fast_for_them(plan, size, direct, padded, small, big):
    # within a fifth of the fastest, what the cost rule is good for
    us = {DIRECT: direct, PADDED: padded, REGS_SMALL: small, REGS_BIG: big}
    form = plan(*size, False)[0]
    assert us[form] <= 1.2 * min(v for v in us.values() if v is not None), (form, us)


def test_every_form_is_listed():
    listed = {(f, p, i) for _, f, p, i in FORMS}
    tiles = {(f, p, None) for f in range(6) for p in (False, True)} | {(PADDED, p, f) for f in range(6) for p in (False, True)}
    assert listed == tiles | {(f, False, None) for f in (DIRECT, ONE_TOKEN, REGS_BIG, REGS_SMALL)}


DEV = torch.device("cuda:0")
u, U, TINY = 2.0 ** -24, {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}, 2.0 ** -24


@pytest.mark.gpu
@pytest.mark.parametrize("size,form,parts,inner", FORMS)
def test_forms(size, form, parts, inner):
    print(f"[q8 forms] {size} form {form} parts {parts} inner {inner}", file=sys.stderr, flush=True)
    T, N, K = size
    g = torch.Generator(device=DEV).manual_seed(T + N + K)
    xq = torch.randint(-127, 128, (T, K), generator=g, device=DEV, dtype=torch.int8)
    wq = torch.randint(-127, 128, (N, K), generator=g, device=DEV, dtype=torch.int8)
    xs, ws = (torch.rand(n, generator=g, device=DEV) * 0.01 + 1e-3 for n in (T, N))
    gm, bias = 1 + 0.3 * torch.randn(N, generator=g, device=DEV), torch.randn(N, generator=g, device=DEV)
    base = ((xq.double() @ wq.double().t()) * xs.double()[:, None]) * ws.double()
    for dt, adapter in ((torch.bfloat16, True), (torch.float32, False), (torch.float16, True)):
        lora = torch.randn(T, N, generator=g, device=DEV).to(dt) if adapter else None
        y = D.matmul_q8(xq, xs, wq, ws, dt, bias=bias, g=gm if adapter else None, lora_out=lora, s=0.5)
        ref, size_of = base + bias.double(), base.abs() + bias.double().abs()
        if adapter:
            extra = gm.double() * 0.5 * lora.double()
            ref, size_of = ref + (gm.double() - 1) * base + extra, size_of + ((gm.double() - 1) * base).abs() + extra.abs()
        bad = ~((y.double() - ref).abs() <= 8 * u * size_of + U[dt] * ref.abs() + TINY)
        assert not bool(bad.any()), (size, dt, int(bad.sum()), bad.nonzero()[:4].tolist())


@pytest.mark.gpu
@pytest.mark.parametrize("N,K", [(512, 2048), (301, 1003), (5120, 5120)])
@pytest.mark.parametrize("dt", [torch.float16, torch.float32])
def test_rows_do_not_depend_on_the_batch(N, K, dt):
    """Bitwise: the sum is exact and every form ends in the same fp32 steps and
    one conversion (fp16: none of them may join the last step with it)."""
    print(f"[q8 forms] batches {N}x{K} {dt}", file=sys.stderr, flush=True)
    g = torch.Generator(device=DEV).manual_seed(N + K)
    xq = torch.randint(-127, 128, (700, K), generator=g, device=DEV, dtype=torch.int8)
    wq = torch.randint(-127, 128, (N, K), generator=g, device=DEV, dtype=torch.int8)
    xs, ws = (torch.rand(n, generator=g, device=DEV) * 0.01 + 1e-3 for n in (700, N))
    gm, bias = 1 + 0.3 * torch.randn(N, generator=g, device=DEV), torch.randn(N, generator=g, device=DEV)
    lora = torch.randn(700, N, generator=g, device=DEV).to(dt)
    for adapter in (True, False):
        y = D.matmul_q8(xq, xs, wq, ws, dt, bias=bias, g=gm if adapter else None, lora_out=lora if adapter else None, s=1.7)
        for lo, hi in ((0, 1), (3, 7), (10, 40), (100, 170), (200, 500)):
            part = D.matmul_q8(xq[lo:hi].contiguous(), xs[lo:hi].contiguous(), wq, ws, dt, bias=bias, g=gm if adapter else None,
                               lora_out=lora[lo:hi].contiguous() if adapter else None, s=1.7)
            torch.cuda.synchronize()
            assert torch.equal(part, y[lo:hi]), (adapter, lo, hi)
