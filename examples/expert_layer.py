"""A layer y = W_shared x + W_expert(x) x, trained: every token goes through shared weights
and those of its own expert.

The tokens are sorted by expert, so that each expert's are a run of rows.  Both products
and the input gradients multiply 8-bit floats with a scale for each block of 128; so does the
shared weights' gradient, from x and dy quantised once more along the tokens.  The
experts' weight gradients are 16-bit products over each expert's own rows.  The weights are
quantised from their binary32 master copies in each step.

    python3 examples/expert_layer.py [--tokens 512] [--channels 1024] [--outputs 768] [--experts 8] [--steps 20]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import matrix_core_gemm_amd as mcg  # noqa: E402

B = 128  # values under one scale


def blocks(n):
    return -(-n // B)


class ExpertLayer:
    """Buffers of one layer for T tokens and G experts: K input channels, N outputs (a multiple
    of 128, so that the experts' weights are quantised as one matrix of G * N rows)."""

    def __init__(self, T, K, N, G, seed=0):
        assert N % B == 0, "outputs: a multiple of 128"
        g = torch.Generator().manual_seed(seed)
        self.T, self.K, self.N, self.G = T, K, N, G
        self.w = (torch.randn(G, N, K, generator=g) / K ** 0.5).cuda()  # master weights: the experts'
        self.ws = (torch.randn(N, K, generator=g) / K ** 0.5).cuda()    # and the shared ones
        f32, bf16 = dict(device="cuda"), dict(dtype=torch.bfloat16, device="cuda")
        u8 = dict(dtype=torch.uint8, device="cuda")
        self.qw, self.sw = torch.empty(G, N, K, **u8), torch.empty(G, N // B, blocks(K), **f32)
        self.qws, self.sws = torch.empty(N, K, **u8), torch.empty(N // B, blocks(K), **f32)
        # x and dy by rows, and along the tokens
        self.qx, self.sx = torch.empty(T, K, **u8), torch.empty(T, blocks(K), **f32)
        self.qxt, self.sxt = torch.empty(T, K, **u8), torch.empty(blocks(T), K, **f32)
        self.qdy, self.sdy = torch.empty(T, N, **u8), torch.empty(T, blocks(N), **f32)
        self.qdyt, self.sdyt = torch.empty(T, N, **u8), torch.empty(blocks(T), N, **f32)
        self.y, self.x, self.dy = torch.empty(T, N, **bf16), torch.empty(T, K, **bf16), None
        self.dx = torch.empty(T, K, **bf16)
        self.dw, self.dws = torch.empty(G, N, K, **f32), torch.empty(N, K, **f32)

    def sort(self, expert):
        """The order of the tokens by expert, and where each expert's rows begin."""
        self.order = torch.argsort(expert, stable=True)
        self.offsets = torch.searchsorted(expert[self.order], torch.arange(self.G + 1, device="cuda")).int()

    def unsorted(self, rows):
        out = torch.empty_like(rows)
        out[self.order] = rows
        return out

    def forward(self, x, expert):
        """x: T x K bf16; expert: T integers below G."""
        T, K, N, G = self.T, self.K, self.N, self.G
        kb, nb = blocks(K), blocks(N)
        self.sort(expert)
        x = x[self.order]
        mcg.quantize_blocks("f32", "e4m3", B, B, G * N, K, self.w, K, self.qw, K, self.sw, kb)
        mcg.quantize_blocks("f32", "e4m3", B, B, N, K, self.ws, K, self.qws, K, self.sws, kb)
        mcg.quantize_blocks("bf16", "e4m3", 1, B, T, K, x, K, self.qx, K, self.sx, kb)
        mcg.quantize_blocks("bf16", "e4m3", B, 1, T, K, x, K, self.qxt, K, self.sxt, K)
        mcg.gemm_grouped_f8_blocks("e4m3", "e4m3", "k_contig", G, T, N, K, self.offsets, self.qx, K, self.sx, kb, self.qw, K, N * K,
                                   self.sw, kb, nb * kb, self.y, N, "bf16")
        mcg.gemm_f8_blocks("e4m3", "e4m3", "k_contig", "k_contig", B, T, N, K, self.qx, K, self.sx, kb, self.qws, K, self.sws, kb,
                           self.y, self.y, N, "bf16", 1.0)
        return self.unsorted(self.y)

    def backward(self, dy):
        """Gradients of the weights (dw, dws) and the input, from the 8-bit tensors and dy."""
        T, K, N, G = self.T, self.K, self.N, self.G
        kb, nb = blocks(K), blocks(N)
        self.dy = dy = dy[self.order]
        mcg.quantize_blocks("bf16", "e5m2", 1, B, T, N, dy, N, self.qdy, N, self.sdy, nb)
        mcg.quantize_blocks("bf16", "e5m2", B, 1, T, N, dy, N, self.qdyt, N, self.sdyt, N)
        # dx = dy . W, of the experts' and the shared weights
        mcg.gemm_grouped_f8_blocks("e5m2", "e4m3", "mn_contig", G, T, K, N, self.offsets, self.qdy, N, self.sdy, nb, self.qw, K, N * K,
                                   self.sw, kb, nb * kb, self.dx, K, "bf16")
        mcg.gemm_f8_blocks("e5m2", "e4m3", "k_contig", "mn_contig", B, T, K, N, self.qdy, N, self.sdy, nb, self.qws, K, self.sws, kb,
                           self.dx, self.dx, K, "bf16", 1.0)
        # dW = dy^T . x, over each expert's rows and over all
        mcg.dequantize_blocks("e4m3", "bf16", 1, B, T, K, self.qx, K, self.sx, kb, self.x, K)
        mcg.gemm_grouped_grad("bf16", G, N, K, T, self.offsets, dy, N, self.x, K, None, self.dw, K, N * K, "f32")
        mcg.gemm_f8_blocks("e5m2", "e4m3", "mn_contig", "mn_contig", 1, N, K, T, self.qdyt, N, self.sdyt, N, self.qxt, K, self.sxt, K,
                           None, self.dws, K, "f32")
        return self.unsorted(self.dx)

    def step(self, rate):
        self.w.add_(self.dw, alpha=-rate)
        self.ws.add_(self.dws, alpha=-rate)


def train(T=512, K=1024, N=768, G=8, steps=20, rate=0.1):
    """The losses of `steps` gradient steps towards a random layer's outputs."""
    g = torch.Generator(device="cuda").manual_seed(1)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")
    x, expert = randn(T, K).bfloat16(), torch.randint(G, (T,), generator=g, device="cuda")
    w, ws = randn(G, N, K) / K ** 0.5, randn(N, K) / K ** 0.5
    target = x.float() @ ws.T
    for e in range(G):
        target[expert == e] += x[expert == e].float() @ w[e].T
    layer, losses = ExpertLayer(T, K, N, G), []
    for _ in range(steps):
        diff = layer.forward(x, expert).float() - target
        losses.append(float(0.5 * diff.square().sum(1).mean()))
        layer.backward((diff / T).bfloat16())
        layer.step(rate)
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--channels", type=int, default=1024)
    ap.add_argument("--outputs", type=int, default=768)
    ap.add_argument("--experts", type=int, default=8)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--rate", type=float, default=0.1)
    a = ap.parse_args()
    for i, loss in enumerate(train(a.tokens, a.channels, a.outputs, a.experts, a.steps, a.rate)):
        print(f"step {i:3d}  loss {loss:.4f}")
