"""Calls run on their operands' GPU: the library launches on the current one,
and the default stream's handle is the same on all of them.  On the CPU, with
the library replaced by a record of what reaches it."""
import types

import pytest
import torch

import dora_adapter_factored_amd as D
from dora_adapter_factored_amd import binding as Bn
from dora_adapter_factored_amd import eightbit as E8


def bf16(*shape):
    return torch.ones(*shape, dtype=torch.bfloat16)


def f32(*shape):
    return torch.ones(*shape)


def codes(*shape):
    return torch.ones(*shape, dtype=torch.int8)


ENTRY_POINTS = {
    "dora_factored_norm": lambda: D.factored_norm(bf16(64, 64), bf16(8, 64), bf16(64, 8), 1.0),
    "dora_factored_norm_noalloc": lambda: D.factored_norm_noalloc(bf16(64, 64), bf16(8, 64), bf16(64, 8), 1.0),
    "dora_factored_norm_group": lambda: D.factored_norm_group([(bf16(64, 64), bf16(8, 64), bf16(64, 8), 1.0, None)]),
    "dora_merge": lambda: D.merge(bf16(64, 64), bf16(8, 64), bf16(64, 8), f32(64), 1.0),
    "dora_compose": lambda: D.compose(bf16(4, 64), bf16(4, 64), f32(64), 1.0),
    "dora_compose_backward": lambda: D.compose_backward(bf16(4, 64), bf16(4, 64), bf16(4, 64), f32(64), f32(64), 1.0),
    "dora_compose_dual": lambda: D.compose_dual(bf16(4, 64), bf16(4, 64), f32(64), 1.0),
    "dora_compose_backward_inner": lambda: D.compose_backward_inner(bf16(4, 64), bf16(4, 64), f32(64), f32(64), 1.0),
    "dora_rmsnorm": lambda: D.rmsnorm(bf16(4, 64), bf16(64), 1e-6),
    "dora_rmsnorm_backward": lambda: D.rmsnorm_backward(bf16(4, 64), bf16(4, 64), bf16(64), f32(4)),
    "dora_quantize_rows": lambda: D.quantize_rows(bf16(4, 64)),
    "dora_dequantize_rows": lambda: D.dequantize_rows(codes(4, 64), f32(4), torch.bfloat16),
    "dora_matmul_q8": lambda: D.matmul_q8(codes(4, 64), f32(4), codes(64, 64), f32(64)),
}


@pytest.mark.parametrize("name", ENTRY_POINTS)
@pytest.mark.parametrize("current", [0, 1])
def test_calls_run_on_their_operands_gpu(monkeypatch, name, current):
    real, on, now = Bn.load(), [], [current]

    class Stub:
        def __getattr__(self, attr):
            if attr.endswith("workspace_size"):
                return getattr(real, attr)
            return lambda *args: on.append((attr, now[0])) or 0

    class device:
        def __init__(self, dev):
            self.dev = dev

        def __enter__(self):
            self.old, now[0] = now[0], 1 if self.dev.index is None else self.dev.index

        def __exit__(self, *exc):
            now[0] = self.old

    # the tensors stand for those of GPU 1: a CPU tensor's device has no index
    call = getattr(Bn, "_call", None)
    if call is not None:
        for mod in (Bn, E8):
            monkeypatch.setattr(mod, "_call", lambda n, dev, *args: call(n, types.SimpleNamespace(type="cuda", index=1), *args))
        monkeypatch.setattr(Bn, "_current_device", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "device", device)
    for mod in (Bn, E8):
        monkeypatch.setattr(mod, "load", lambda: Stub())
        monkeypatch.setattr(mod, "_stream", lambda dev: 0)
    ENTRY_POINTS[name]()
    assert on == [(name, 1)] and now == [current]


def test_every_entry_point_is_here():
    launching = {n for n, (_, args) in Bn._SIGNATURES.items() if n.startswith("dora_") and args and args[-1] is Bn._vp}
    assert launching == set(ENTRY_POINTS)
