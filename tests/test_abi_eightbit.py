"""Refusals of the 8-bit entry points, on the host before any launch (no GPU
needed: every call here returns from validation or asks for no rows)."""
import ctypes

import pytest
import torch

import dora_adapter_factored_amd as D
from dora_adapter_factored_amd import binding as Bn

FAKE = ctypes.c_void_p(0x10000)
OTHER = ctypes.c_void_p(0x20000)
THIRD = ctypes.c_void_p(0x30000)
WS = ctypes.c_void_p(0x100000)
INV, UNS, WSP = Bn.DORA_ERR_INVALID_ARG, Bn.DORA_ERR_UNSUPPORTED, Bn.DORA_ERR_WORKSPACE
BIG = 1 << 31


@pytest.fixture(scope="module")
def lib():
    return D.load()


def call(fn, defaults, **kw):
    assert set(kw) <= set(defaults)
    return fn(*{**defaults, **kw}.values())


NORM = dict(x=FAKE, residual=OTHER, w=FAKE, eps=1e-6, T=4, d=8, dtype=1, h=OTHER, y=THIRD, q=None, qscale=None, rstd=None,
            stream=None)


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(w=None), dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(T=-1),
    dict(T=BIG), dict(d=0), dict(d=BIG), dict(dtype=3), dict(dtype=-1), dict(q=FAKE), dict(qscale=FAKE),
    dict(h=None, y=None), dict(y=FAKE), dict(y=OTHER),
])
def test_rmsnorm_refuses(lib, kw):
    assert call(lib.dora_rmsnorm, NORM, **kw) == INV
    assert lib.dora_last_error_detail()


BWD = dict(dy=FAKE, h=OTHER, w=FAKE, rstd=FAKE, dh=None, T=4, d=8, dtype=1, dx=THIRD, dw=FAKE, ws=WS, nbytes=1 << 20,
           stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(dy=None), INV), (dict(h=None), INV), (dict(w=None), INV), (dict(rstd=None), INV), (dict(dx=None), INV),
    (dict(dx=OTHER), INV), (dict(T=-1), INV), (dict(d=0), INV), (dict(dtype=9), INV), (dict(ws=None), WSP),
    (dict(nbytes=16), WSP), (dict(ws=ctypes.c_void_p(0x100010)), WSP),
])
def test_rmsnorm_backward_refuses(lib, kw, status):
    assert call(lib.dora_rmsnorm_backward, BWD, **kw) == status


QUANT = dict(x=FAKE, col_scale=None, n=4, d=8, dtype=1, q=OTHER, scale=THIRD, stream=None)
DEQ = dict(q=FAKE, scale=OTHER, n=4, d=8, dtype=1, out=THIRD, stream=None)


@pytest.mark.parametrize("kw", [dict(n=-1), dict(n=BIG), dict(d=0), dict(d=BIG), dict(dtype=7), dict(q=None),
                                dict(scale=None)])
def test_row_quantisation_refuses(lib, kw):
    assert call(lib.dora_quantize_rows, QUANT, **kw) == INV
    assert call(lib.dora_dequantize_rows, DEQ, **kw) == INV


def test_row_quantisation_refuses_missing_rows(lib):
    assert call(lib.dora_quantize_rows, QUANT, x=None) == INV
    assert call(lib.dora_dequantize_rows, DEQ, out=None) == INV


MM = dict(xq=FAKE, xs=FAKE, wq=OTHER, ws=FAKE, bias=None, g=None, lora=None, s=1.0, T=4, N=8, K=16, dtype=1, y=THIRD,
          wsp=WS, nbytes=1 << 40, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(xq=None), INV), (dict(xs=None), INV), (dict(wq=None), INV), (dict(y=None), INV), (dict(g=FAKE), INV),
    (dict(lora=FAKE), INV), (dict(s=float("nan")), INV), (dict(T=-1), INV), (dict(T=BIG), INV), (dict(N=0), INV),
    (dict(N=BIG), INV), (dict(N=(1 << 24) + 1), UNS), (dict(K=0), INV), (dict(K=131072), UNS), (dict(dtype=4), INV), (dict(y=FAKE), INV),
    (dict(y=OTHER), INV),
])
def test_matmul_q8_refuses(lib, kw, status):
    assert call(lib.dora_matmul_q8, MM, **kw) == status


def test_workspace_queries(lib):
    n = ctypes.c_size_t()
    assert lib.dora_matmul_q8_workspace_size(4, 8, 131072, ctypes.byref(n)) == UNS
    assert lib.dora_matmul_q8_workspace_size(4, 8, 16, None) == INV
    assert lib.dora_matmul_q8_workspace_size(-1, 8, 16, ctypes.byref(n)) == INV
    assert lib.dora_rmsnorm_backward_workspace_size(4, 0, ctypes.byref(n)) == INV
    assert lib.dora_rmsnorm_backward_workspace_size(4, 8, None) == INV
    for T in (1, 7, 2048, 1 << 20):   # partial rows of dw stay few
        assert lib.dora_rmsnorm_backward_workspace_size(T, 5120, ctypes.byref(n)) == 0
        assert n.value <= 512 * 5120 * 4


def test_workspaces_follow_the_forms():
    # tiles that leave CUs idle are taken in parts, whose sums the workspace
    # holds; a full chip and one token need none; odd rows are padded in it
    assert D.matmul_q8_workspace_size(24, 5120, 5120) >= 2 * 24 * 5120 * 4
    assert D.matmul_q8_workspace_size(333, 5120, 27648) >= 2 * 333 * 5120 * 4
    assert D.matmul_q8_workspace_size(2048, 8192, 8192) == 0 and D.matmul_q8_workspace_size(1, 8192, 8191) == 0
    assert (2000 + 4099) * 4099 <= D.matmul_q8_workspace_size(2000, 4099, 4099) <= (2000 + 4099 + 2) * 4112 + 512


def test_a_small_workspace_is_refused(lib):
    need = ctypes.c_size_t()
    for T, N, K in ((64, 1024, 8192), (200, 1024, 8192), (333, 4090, 2056), (2048, 5120, 5120)):
        assert lib.dora_matmul_q8_workspace_size(T, N, K, ctypes.byref(need)) == 0
        if need.value:
            assert call(lib.dora_matmul_q8, MM, T=T, N=N, K=K, nbytes=need.value - 1) == WSP
            assert call(lib.dora_matmul_q8, MM, T=T, N=N, K=K, wsp=None) == WSP


def test_the_binding_refuses_what_the_library_cannot_see():
    x, w = torch.zeros(4, 8), torch.zeros(8)
    with pytest.raises(ValueError):
        D.rmsnorm(torch.zeros(8), w, 1e-6)                       # one dimension
    with pytest.raises(ValueError):
        D.rmsnorm(x.t(), torch.zeros(4), 1e-6)                   # not contiguous
    with pytest.raises(ValueError):
        D.rmsnorm(x, w.bfloat16(), 1e-6)                         # another dtype
    with pytest.raises(ValueError):
        D.rmsnorm(x, w, 1e-6, torch.zeros(4, 9))                 # another shape
    with pytest.raises(ValueError):
        D.rmsnorm(x, w, 1e-6, h=torch.zeros(4, 8))               # h without a residual
    with pytest.raises(ValueError):
        D.rmsnorm_q8(x, w, 1e-6, q=torch.zeros(4, 8))            # codes that are not int8
    with pytest.raises(ValueError):
        D.quantize_rows(x.double())
    with pytest.raises(TypeError):
        D.quantize_rows([1.0])
    with pytest.raises(ValueError):
        D.quantize_rows(x, torch.zeros(7))
    with pytest.raises(ValueError):
        D.dequantize_rows(x, torch.zeros(4), torch.float32)      # not int8
    q, s = torch.zeros(4, 8, dtype=torch.int8), torch.zeros(4)
    wq, ws = torch.zeros(6, 8, dtype=torch.int8), torch.zeros(6)
    for bad in (dict(xq=x), dict(wq=torch.zeros(6, 9, dtype=torch.int8)), dict(xscale=torch.zeros(5)),
                dict(wscale=torch.zeros(5)), dict(bias=torch.zeros(5)), dict(g=torch.zeros(6)),
                dict(lora_out=torch.zeros(4, 6)), dict(g=torch.zeros(6), lora_out=torch.zeros(4, 6)),   # lora_out not bf16
                dict(dtype=torch.float64), dict(out=torch.zeros(4, 6))):
        with pytest.raises(ValueError):
            D.matmul_q8(**{**dict(xq=q, xscale=s, wq=wq, wscale=ws), **bad})
