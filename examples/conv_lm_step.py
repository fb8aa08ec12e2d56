"""Train a small causal convolution language model on one GB300 with this package's gradients and updates.

    python examples/conv_lm_step.py [--steps 30]

Tokens are looked up (wg_embedding_lookup), pass through residual blocks of a causal 1-D convolution, and are scored
against the same table (wg_linear).  Per step the library computes the blocks' activations and residuals
(wg_activation) and their gradients (wg_activation_bwd), each convolution's weight gradient (wg_conv_bwd_weight) and
input gradient (wg_conv_bwd_data), the scores' gradients (wg_linear_bwd_data, wg_linear_bwd_weight), the table's gradient
as it was looked up (wg_embedding_bwd_weight, added to what the scores leave there), and the convolutions'
orthogonalised update (wg_muon_update: momentum, Newton-Schulz products, weights).  torch computes what the library has
no operator for: the convolutions' forward pass and the loss.  The data are sequences in which every token follows from
the two before it.
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from implicit_gemm_gb300 import binding, build  # noqa: E402


class CausalConv:
    """y[n, l, k] = sum over x, c of w[k, x, c] u[n, l - (X - 1) + x, c]; gradients and update by the library."""

    def __init__(self, batch, length, channels, taps, gen):
        self.spec = {"ndim": 1, "G": 1, "N": batch, "C": channels, "K": channels, "in": [length], "filt": [taps],
                     "stride": [1], "dil": [1], "pad_l": [taps - 1], "pad_r": [0], "in_dtype": "bf16",
                     "out_dtype": "fp32"}
        fan = taps * channels
        self.w = (torch.randn((1, channels, taps, channels), generator=gen, device="cuda") / math.sqrt(fan)).bfloat16()
        self.momentum = torch.zeros(self.w.shape, device="cuda")
        self.muon = {"rows": channels, "cols": fan, "grad_dtype": "fp32", "weight_dtype": "bf16", "momentum": 0.9,
                     "lr": 0.05, "scale": 0.2}

    def forward(self, u):
        self.u = u
        w = self.w[0].permute(0, 2, 1)  # (K, C, X)
        return F.conv1d(F.pad(u.mT, (self.spec["filt"][0] - 1, 0)), w).mT.contiguous()

    def backward(self, dy):
        self.dw = binding.conv_bwd_weight(self.spec, self.u, dy)
        return binding.conv_bwd_data(self.spec, dy, self.w)

    def update(self):
        binding.muon_update(self.muon, self.dw, momentum=self.momentum, weight=self.w)


class ConvLM:
    def __init__(self, batch=16, length=128, vocab=512, channels=64, taps=4, layers=2, seed=0):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        self.vocab, self.channels = vocab, channels
        self.table = torch.randn((vocab, channels), generator=gen, device="cuda") / math.sqrt(channels)
        self.layers = [CausalConv(batch, length, channels, taps, gen) for _ in range(layers)]
        self.scale = math.sqrt(channels)
        self.m1, self.m2, self.t = torch.zeros_like(self.table), torch.zeros_like(self.table), 0

    def gradients(self, tokens, targets):
        """The loss; leaves each convolution's dw and the table's gradient behind."""
        h = binding.embedding_lookup(tokens, self.table, self.scale)  # (N, L, C), fp32
        kept = []
        for layer in self.layers:
            y = layer.forward(h.bfloat16())
            kept.append(y)
            h = binding.activation(y, residual=h, activation="gelu")  # y in bf16, h in fp32
        flat, table = h.reshape(-1, self.channels).bfloat16(), self.table.bfloat16()
        rows = len(flat)
        scores = binding.linear(flat, table, out=torch.empty((rows, self.vocab), device="cuda"))
        loss = F.cross_entropy(scores, targets.reshape(-1))
        d = torch.softmax(scores, -1)
        d[torch.arange(rows, device="cuda"), targets.reshape(-1)] -= 1.0
        d = d.bfloat16()  # (of the loss's sum over the rows: the mean's would lose bits in 16)
        self.dtable = binding.linear_bwd_weight(flat, d) / rows
        dh = (binding.linear_bwd_data(d, table, out=torch.empty(flat.shape, device="cuda")) / rows).view_as(h)
        for layer, y in zip(reversed(self.layers), reversed(kept)):
            dy = binding.activation_bwd(dh, y, activation="gelu")
            dh = dh + layer.backward(dy).view_as(dh)
        binding.embedding_bwd_weight(tokens, dh.contiguous(), self.vocab, self.scale, out=self.dtable, accumulate=True)
        return loss

    def update(self):
        for layer in self.layers:
            layer.update()
        self.t += 1  # Adam for the table
        self.m1.lerp_(self.dtable, 0.1)
        self.m2.lerp_(self.dtable.square(), 0.01)
        step = (self.m1 / (1 - 0.9 ** self.t)) / ((self.m2 / (1 - 0.99 ** self.t)).sqrt() + 1e-8)
        self.table -= 0.01 * step


def batch_of(gen, n, length, vocab):
    seq = torch.randint(vocab, (n, 2), generator=gen, device="cuda")
    cols = [seq[:, 0], seq[:, 1]]
    for _ in range(length - 1):
        cols.append((3 * cols[-1] + cols[-2] + 7) % vocab)
    seq = torch.stack(cols, 1)
    return seq[:, :length].contiguous(), seq[:, 1:length + 1].contiguous()


def main(steps=30, seed=0, say=print):
    build.build()
    model = ConvLM(vocab=64, seed=seed)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed + 1)
    losses = []
    for i in range(steps):
        tokens, targets = batch_of(gen, 16, 128, 64)
        loss = model.gradients(tokens, targets)
        model.update()
        losses.append(float(loss))
        if i % 5 == 0 or i == steps - 1:
            say(f"step {i:3d}  loss {losses[-1]:.4f}")
    binding.wg_check_status()
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=30)
    main(ap.parse_args().steps)
