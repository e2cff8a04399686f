"""The row operators where the other tests do not reach: pointers off 16 bytes
with rows that are whole packs.  The arithmetic is the same in the same order, so
results are equal."""
import sys

import pytest
import torch

import dora_adapter_factored_amd as D
from test_eightbit import DEV, DT, misaligned, randn, rng

pytestmark = pytest.mark.gpu


def say(*a):
    print(*a, file=sys.stderr, flush=True)


# register forms of one, two, four and the most packs a thread, and rows too long for them
ROWS = [(9, 512), (600, 2048), (600, 8192), (520, 9216), (3, 28672), (3, 70000)]


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
