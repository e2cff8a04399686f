"""Codes and scales bit for bit those of the stated formulas in fp32:
scale = max|p| * fl(1/127), code = rint(fl(p / scale)), evaluated by numpy on
the host, whose fp32 division is correctly rounded.  p = x * col_scale is one
fp32 product.  Equality: no tolerance."""
import sys

import numpy as np
import pytest
import torch

import dora_adapter_factored_amd as D

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def definition(p):
    p = np.asarray(p, np.float32)
    scale = np.max(np.abs(p), axis=1) * np.float32(1 / 127)
    assert scale.dtype == np.float32
    quot = np.divide(p, scale[:, None], out=np.zeros_like(p), where=scale[:, None] > 0)
    return np.rint(quot).astype(np.int8), scale


def check(x, col_scale=None):
    q, scale = D.quantize_rows(x, col_scale)
    torch.cuda.synchronize()
    p = x.float().cpu().numpy()
    if col_scale is not None:
        p = p * col_scale.cpu().numpy()
    want, ws = definition(p)
    assert np.array_equal(scale.cpu().numpy().view(np.uint32), ws.view(np.uint32))
    assert np.array_equal(q.cpu().numpy(), want)


@pytest.mark.parametrize("n,d", [(300, 2056), (600, 1003), (5, 70000)])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_codes_are_the_formulas(n, d, dt):
    say(f"[codes] {n}x{d} {dt}")
    g = torch.Generator(device=DEV).manual_seed(n + d)
    x = torch.randn(n, d, generator=g, device=DEV)
    if dt != "f16":   # rows of every size: 2^-90 to 2^90
        x = x * torch.exp2(torch.randint(-90, 91, (n, 1), generator=g, device=DEV).float())
    x = x.to(DT[dt])
    check(x)
    check(x, torch.rand(d, generator=g, device=DEV) + 0.5)


def test_codes_next_to_ties():
    # values within three units in the last place of (k + 1/2) scale
    say("[codes] ties")
    rng = np.random.default_rng(5)
    top = (1 + rng.random(2000)).astype(np.float32) * np.exp2(rng.integers(-90, 90, 2000)).astype(np.float32)
    scale = top * np.float32(1 / 127)
    k = np.arange(127) + 0.5
    near = (k[None, :] * scale.astype(np.float64)[:, None]).astype(np.float32)
    x = np.concatenate([top[:, None]] + [(near.view(np.int32) + i).view(np.float32) for i in range(-3, 4)], axis=1)
    x = np.minimum(x, top[:, None]) * np.where(rng.random(x.shape) < 0.5, -1, 1).astype(np.float32)
    x[:, 0] = top
    check(torch.from_numpy(np.ascontiguousarray(x)).to(DEV))
