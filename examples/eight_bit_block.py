"""An MLP block whose frozen weights are held in 8 bits, with DoRA adapters:
decoding, a prompt, and one training step.

    python examples/eight_bit_block.py [--hidden 4096] [--inner 8192] [--rank 16] [--tokens 512]

Serving: residual and norm go to 8 bits in one call (rmsnorm_q8), the up
projection takes its adapter unmerged in the product's own call, the down
projection has its adapter merged (factored_norm, merge) before it is quantised.
Training: the frozen weight is a LinearQ8, the adapter's two products are plain
bf16, the composition is DoRACompose and the norm RMSNorm; gradients reach x,
the norm's weight, A, B and m.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import dora_adapter_factored_amd as D  # noqa: E402
import dora_inputs as DI  # noqa: E402

EPS = 1e-6


def projection(d_out, d_in, r, seed, dev):
    """A frozen projection with a DoRA adapter."""
    return DI.make_layer(DI.custom_spec(d_out, d_in, r, 1, dtype="bf16", s=2.0, b_std=0.02, m_noise=0.05), seed, device=dev,
                         activations=False, gen_device=dev)


class Block:
    def __init__(self, hidden, inner, r, dev):
        self.up, self.down = projection(inner, hidden, r, 1, dev), projection(hidden, inner, r, 2, dev)
        self.norm_w = torch.ones(hidden, dtype=torch.bfloat16, device=dev)
        # 8-bit weights, laid out once: W0 with the adapter beside it, the other merged
        self.up_q, self.up_s = D.quantize_rows(self.up.W0)
        self.up_qt = self.up_q.t().contiguous()
        # the norm of the weight that the product computes with, which is the one in 8 bits
        W8 = D.dequantize_rows(self.up_q, self.up_s, torch.float32)
        self.up_wnorm, self.up_g = D.factored_norm(W8, self.up.A.float(), self.up.B.float(), self.up.spec.s, self.up.m)
        _, g = D.factored_norm(self.down.W0, self.down.A, self.down.B, self.down.spec.s, self.down.m)
        self.down_q, self.down_s = D.quantize_rows(D.merge(self.down.W0, self.down.A, self.down.B, g, self.down.spec.s))

    def serve(self, x, residual):
        """(output, new residual) for the tokens x [T, hidden]."""
        y = torch.empty_like(x)   # the adapter's branch reads the norm's output itself
        q, scale, h = D.rmsnorm_q8(x, self.norm_w, EPS, residual, y=y)
        lora = (y @ self.up.A.t()) @ self.up.B.t()
        u = D.matmul_q8(q, scale, self.up_q, self.up_s, g=self.up_g, lora_out=lora, s=self.up.spec.s)
        return D.linear_q8(torch.nn.functional.silu(u), self.down_q, self.down_s), h

    def plain(self, x, residual):
        """The same in fp32 with unquantised weights."""
        h = x.float() + residual.float()
        y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS) * self.norm_w.float()

        def dora(v, L):
            W = L.W0.float() + L.spec.s * (L.B.float() @ L.A.float())
            return v @ (W * (L.m / W.norm(dim=1))[:, None]).t()

        return dora(torch.nn.functional.silu(dora(y, self.up)), self.down), h

    def train_step(self, x, residual, target):
        """Loss and gradients of one step through the norm and the up projection."""
        leaf = lambda t: t.detach().clone().requires_grad_()  # noqa: E731
        x, A, B, m, w = leaf(x), leaf(self.up.A), leaf(self.up.B), leaf(self.up.m), leaf(self.norm_w)
        y, h = D.RMSNorm.apply(x, residual, w, EPS)
        base = D.LinearQ8.apply(y, self.up_q, self.up_s, self.up_qt)
        lora = (y @ A.t()) @ B.t()
        out = D.DoRACompose.apply(base, lora, m, self.up_g, self.up_wnorm, self.up.spec.s, D.default_eps(torch.bfloat16))
        loss = (out.float() - target.float()).square().mean() + h.float().square().mean()
        loss.backward()
        return loss.detach(), {"x": x.grad, "norm_w": w.grad, "A": A.grad, "B": B.grad, "m": m.grad}


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--inner", type=int, default=8192)
    ap.add_argument("--rank", type=int, default=16)
    ap.add_argument("--tokens", type=int, default=512)
    a = ap.parse_args(argv)
    dev = torch.device("cuda:0")
    torch.manual_seed(0)
    block = Block(a.hidden, a.inner, a.rank, dev)
    off = {}
    for T in (1, a.tokens):
        x, res = (torch.randn(T, a.hidden, device=dev).bfloat16() for _ in range(2))
        out, h = block.serve(x, res)
        ref, ref_h = block.plain(x, res)
        off[T] = float((out.float() - ref).norm() / ref.norm())
        print(f"{T} tokens: output {tuple(out.shape)}, {100 * off[T]:.2f}% from the fp32 block")
    x, res = (torch.randn(a.tokens, a.hidden, device=dev).bfloat16() for _ in range(2))
    loss, grads = block.train_step(x, res, torch.zeros(a.tokens, a.inner, dtype=torch.bfloat16, device=dev))
    print(f"training step: loss {float(loss):.4f}, gradient norms "
          + ", ".join(f"{k} {float(v.float().norm()):.3g}" for k, v in grads.items()))
    return off, loss, grads


if __name__ == "__main__":
    main()
