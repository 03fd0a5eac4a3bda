"""A layer y = W . norm(h), h = x + r, trained with the 8-bit linear layer.

What a training step keeps between its passes is 8-bit: the normed input (the codes
that the product reads anyway) and the residual stream before the norm (a checkpoint
of its rows).  The weights are quantised from their binary32 master copy in each step.

    python3 examples/linear8_layer.py [--tokens 512] [--channels 1024] [--outputs 768] [--steps 20]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import matrix_core_gemm_amd as mcg  # noqa: E402

EPS = 1e-5


class Linear8:
    """Buffers of one layer for T tokens: K input channels, N outputs, 16-bit activations."""

    def __init__(self, T, K, N, seed=0):
        g = torch.Generator().manual_seed(seed)
        dev = dict(device="cuda")
        self.T, self.K, self.N = T, K, N
        self.w = (torch.randn(N, K, generator=g) / K ** 0.5).cuda()  # master weights
        self.gamma = torch.ones(K, **dev)                            # of the norm
        bf16, i8 = dict(dtype=torch.bfloat16, device="cuda"), dict(dtype=torch.int8, device="cuda")
        self.qw, self.sw = torch.empty(N, K, **i8), torch.empty(N, **dev)   # weights, a scale per output channel
        self.qx, self.sx = torch.empty(T, K, **i8), torch.empty(T, **dev)   # the normed input, a scale per token
        self.qh, self.sh = torch.empty(T, K, **i8), torch.empty(T, **dev)   # the residual stream's checkpoint
        self.h, self.y = torch.empty(T, K, **bf16), torch.empty(T, N, **bf16)
        self.rstd = torch.empty(T, **dev)
        self.dx, self.dh = torch.empty(T, K, **bf16), torch.empty(T, K, **bf16)
        self.dw, self.dgamma = torch.empty(N, K, **dev), torch.empty(K, **dev)
        need = max(mcg.i8_scaled_workspace_bytes("k_contig", T, N, K, self.qx, K, self.qw, K),
                   mcg.grad_i8_workspace_bytes("bf16", "k_contig", T, K, N, self.y, N, self.qw, K, "bf16"),
                   mcg.grad_i8_workspace_bytes("bf16", "mn_contig", N, K, T, self.y, N, self.qx, K, "f32"),
                   mcg.rmsnorm_backward_workspace_bytes(T, K), 16)
        self.ws = torch.empty(need, dtype=torch.uint8, **dev)

    def forward(self, x, r):
        T, K, N = self.T, self.K, self.N
        mcg.quantize_rows("f32", N, K, self.w, K, self.qw, K, self.sw)
        mcg.rmsnorm_quant("bf16", T, K, x, K, r, K, self.gamma.bfloat16(), EPS, self.h, K, self.qx, K, self.sx, self.rstd)
        mcg.quantize_rows("bf16", T, K, self.h, K, self.qh, K, self.sh)
        mcg.gemm_i8_scaled("k_contig", T, N, K, self.qx, K, self.sx, self.qw, K, self.sw, None, self.y, N, "bf16", self.ws)
        return self.y, self.h

    def backward(self, dy, dh_out=None):
        """Gradients of the weights (dw), the norm (dgamma) and the input (dh), from the
        8-bit tensors alone; dh_out: what reaches the residual stream past this layer."""
        T, K, N = self.T, self.K, self.N
        mcg.gemm_grad_i8("bf16", "k_contig", T, K, N, dy, N, self.qw, K, self.sw, None, self.dx, K, "bf16", 0.0, self.ws)
        mcg.gemm_grad_i8("bf16", "mn_contig", N, K, T, dy, N, self.qx, K, self.sx, None, self.dw, K, "f32", 0.0, self.ws)
        mcg.rmsnorm_backward("bf16", "i8", T, K, self.dx, K, self.qh, K, self.sh, self.gamma.bfloat16(), self.rstd,
                             dh_out, 0 if dh_out is None else K, self.dh, K, self.dgamma, self.ws)
        return self.dh

    def step(self, rate):
        self.w.add_(self.dw, alpha=-rate)
        self.gamma.add_(self.dgamma, alpha=-rate)


def train(T=512, K=1024, N=768, steps=20, rate=0.1):
    """The losses of `steps` gradient steps towards a random layer's outputs."""
    g = torch.Generator(device="cuda").manual_seed(1)
    x, r = (torch.randn(T, K, generator=g, device="cuda").bfloat16() for _ in range(2))
    h = x.float() + r.float()
    target = (h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS)) @ (torch.randn(K, N, generator=g, device="cuda") / K ** 0.5)
    layer, losses = Linear8(T, K, N), []
    for _ in range(steps):
        y, _ = layer.forward(x, r)
        diff = y.float() - target
        losses.append(float(0.5 * diff.square().sum(1).mean()))
        layer.backward((diff / T).bfloat16())
        layer.step(rate)
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--channels", type=int, default=1024)
    ap.add_argument("--outputs", type=int, default=768)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--rate", type=float, default=0.1)
    a = ap.parse_args()
    for i, loss in enumerate(train(a.tokens, a.channels, a.outputs, a.steps, a.rate)):
        print(f"step {i:3d}  loss {loss:.4f}")
