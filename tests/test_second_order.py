"""The autograd functions have first gradients only.  A second one has to be
refused: the kernels' results carry no graph, so its terms would be missing
without a word.  On the CPU, with each kernel replaced by its formula."""
import pytest
import torch

import dora_adapter_factored_amd as D
from dora_adapter_factored_amd import binding as Bn
from dora_adapter_factored_amd import eightbit as E8

T, N = 3, 8


def rmsnorm(x, w, eps, residual=None):
    h = x if residual is None else x + residual
    rstd = torch.rsqrt(h.square().mean(1) + eps)
    return h * rstd[:, None] * w, h, rstd


def rmsnorm_backward(dy, h, w, rstd, dh=None, need_dw=True):
    u, r = dy * w, rstd[:, None]
    return r * (u - h * r * r * (u * h).mean(1, keepdim=True)), (dy * h * r).sum(0)


def compose(base, lora, g, s, delta_only=False):
    return base + ((g - 1) * base + g * s * lora)


def compose_backward(dy, base, lora, g, wnorm, s, eps, delta_only, need_d_base, need_d_lora, need_d_m):
    return dy * g, dy * g * s, (dy * (base + s * lora)).sum(0) / wnorm


def compose_dual(base, lora, g, s, delta_only=False):
    return compose(base, lora, g, s), base + s * lora


def compose_backward_inner(dy, inner, g, wnorm, s, eps, delta_only, need_d_base, need_d_lora, need_d_m):
    return dy * g, dy * g * s, (dy * inner).sum(0) / wnorm


def call_norm(x):
    return D.RMSNorm.apply(x, x.detach().clone(), torch.ones(N), 1e-6)[0]


def call_linear(x):
    return D.LinearQ8.apply(x, torch.ones(N, N, dtype=torch.int8), torch.ones(N), torch.ones(N, N, dtype=torch.int8))


def call_compose(x):
    return D.DoRACompose.apply(x, x, torch.ones(N), torch.ones(N), torch.ones(N), 1.0, 1e-6)


def call_inner(x):
    return D.DoRAComposeInner.apply(x, x, torch.ones(N), torch.ones(N), torch.ones(N), 1.0, 1e-6)


@pytest.mark.parametrize("call", [call_norm, call_linear, call_compose, call_inner])
def test_a_second_gradient_is_refused(monkeypatch, call):
    monkeypatch.setattr(E8, "rmsnorm", rmsnorm)
    monkeypatch.setattr(E8, "rmsnorm_backward", rmsnorm_backward)
    monkeypatch.setattr(E8, "linear_q8", lambda x, wq, ws: x @ (wq * ws[:, None]).t())
    monkeypatch.setattr(E8, "linear_q8_backward", lambda dy, wqt, ws: (dy * ws) @ wqt.float().t())
    for f in (compose, compose_backward, compose_dual, compose_backward_inner):
        monkeypatch.setattr(Bn, f.__name__, f)
    x = torch.randn(T, N, generator=torch.Generator().manual_seed(1)).requires_grad_()
    (first,) = torch.autograd.grad(call(x).square().sum(), x, create_graph=True)   # the first gradient as before
    (plain,) = torch.autograd.grad(call(x).square().sum(), x)
    assert torch.equal(first, plain)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        first.square().sum().backward()
