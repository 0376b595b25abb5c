"""Trains one attention block on synthetic data: a batch of small graphs whose nodes have a type and a place.

    x = embed(type);  y = norm(x);  q, k, v = linear(y)
    out = x + dropout(linear(attention(q, k, v, places))),   loss = mean((out - target)^2) / 2

The target is the same block with other weights and without dropout.  One linear layer makes q, k and v side by side; the
attention reads them as columns of its result and writes their gradients into the columns of one tensor.  Both weight
banks take orthogonalised (Muon) steps; the embedding, the norm's weights and the slopes of the distance bias take plain
gradient steps.

    python examples/train_attention.py [--graphs 64] [--channels 64] [--heads 4] [--types 10] [--steps 20]
"""
from __future__ import annotations

import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from equivariant_gnn_tensor_receiver_amd import attention as at  # noqa: E402
from equivariant_gnn_tensor_receiver_amd import layers  # noqa: E402


class Block:
    """The operators, their workspaces' sizes, and the weights, for features of `irreps`."""

    def __init__(self, irreps, heads, types, p, seed, device):
        self.norm = layers.Norm(irreps)
        F = self.norm.features
        self.project = layers.Linear(irreps, "+".join([irreps] * 3), 1)
        self.attention = at.Attention(irreps, irreps, heads)
        self.mix = layers.Linear(irreps, irreps, 1)
        self.dropout = at.Dropout(irreps, p)
        self.embed = at.Embedding(types, F, F ** 0.5)
        gen = torch.Generator(device).manual_seed(seed)
        normal = lambda shape, scale: torch.randn(shape, generator=gen, device=device) * scale  # noqa: E731
        mul = max(shape[0] for shape in (self.mix.block(i)[1] for i in range(self.mix.num_blocks)))
        self.E = normal(self.embed.w_shape, F ** -0.5)
        self.P, self.M = normal(self.project.w_shape, mul ** -0.5), normal(self.mix.w_shape, mul ** -0.5)
        self.gamma = torch.ones(self.norm.num_weights, device=device)
        self.beta = torch.zeros(self.norm.num_biases, device=device)
        self.slope = 2.0 ** -torch.arange(1.0, heads + 1, device=device)
        self.opt_p, self.opt_m = (layers.Muon(layers.weight_blocks(v)) for v in (self.project, self.mix))
        self.mom_p, self.mom_m = torch.zeros_like(self.P), torch.zeros_like(self.M)

    def forward(self, x, batch, rng=None):
        """The block on node features x; rng: (seed, offset) of the dropout, None without one."""
        n = x.shape[0]
        self.x, self.batch, self.rng, self.all = x, batch, rng, layers.Groups(n)
        self.stats = torch.empty(self.norm.stats_shape(n), device=x.device)
        self.y = layers.tpconv_norm_forward(self.norm, x, self.gamma, self.beta, stats=self.stats)
        self.qkv = layers.tpconv_linear_forward(self.project, self.all, self.y, self.P)
        self.saved = torch.empty(self.attention.saved_size(n), device=x.device)
        self.o = at.tpconv_attention_forward(self.attention, batch, *self.qkv.chunk(3, 1), slope=self.slope,
                                             saved=self.saved)
        z = layers.tpconv_linear_forward(self.mix, self.all, self.o, self.M)
        return x + z if rng is None else at.tpconv_dropout_forward(self.dropout, z, rng, residual=x)

    def backward(self, grad_out):
        """The gradient of x; those of the weights, slopes and places stay in the block."""
        gz = grad_out if self.rng is None else at.tpconv_dropout_backward(self.dropout, grad_out, self.rng)
        go, self.grad_m = layers.tpconv_linear_backward(self.mix, self.all, self.o, self.M, gz)
        gqkv = torch.empty_like(self.qkv)
        gq, gk, gv = gqkv.chunk(3, 1)
        *_, self.grad_slope, self.grad_pos, _ = at.tpconv_attention_backward(
            self.attention, self.batch, *self.qkv.chunk(3, 1), self.o, self.saved, go, slope=self.slope,
            want=("slope", "pos"), grad_q=gq, grad_k=gk, grad_v=gv)
        gy, self.grad_p = layers.tpconv_linear_backward(self.project, self.all, self.y, self.P, gqkv)
        gx, self.grad_gamma, self.grad_beta = layers.tpconv_norm_backward(self.norm, self.x, self.gamma, gy,
                                                                          stats=self.stats)
        return gx + grad_out

    def update(self, lr, index, grad_x):
        for opt, w, g, m in ((self.opt_p, self.P, self.grad_p, self.mom_p), (self.opt_m, self.M, self.grad_m, self.mom_m)):
            layers.tpconv_muon_step(opt, w, g, m, lr, W_out=w, momentum_out=m)
        self.E -= lr * at.tpconv_embed_backward(self.embed, index, grad_x)
        self.gamma -= lr * self.grad_gamma
        self.beta -= lr * self.grad_beta
        self.slope -= lr * self.grad_slope


def train(graphs=64, channels=64, heads=4, types=10, steps=20, p=0.1, lr=0.02, seed=0, device="cuda:0"):
    """The loss before every step, and after the last."""
    device = torch.device(device)
    rng = np.random.default_rng(seed)
    sizes = rng.integers(5, 40, graphs)
    n = int(sizes.sum())
    to = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(device)  # noqa: E731
    index = to(rng.integers(0, types, n).astype(np.int32))
    pos = to((rng.random((n, 3)) * np.repeat((20.0 * sizes) ** (1 / 3), sizes)[:, None]).astype(np.float32))
    batch = at.Batch(n, to(np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)), pos)
    block, teacher = (Block(f"{channels}x0e", heads, types, p, s, device) for s in (seed, seed + 1))
    target = teacher.forward(at.tpconv_embed_forward(teacher.embed, index, teacher.E), batch)
    state = torch.tensor([seed, 0], dtype=torch.int64, device=device)
    losses = []
    for step in range(steps + 1):
        x = at.tpconv_embed_forward(block.embed, index, block.E)
        diff = block.forward(x, batch, state) - target
        losses.append(float(diff.square().mean()) / 2)
        if step == steps:
            break
        block.update(lr, index, block.backward(diff / diff.numel()))
        state[1] += 1  # the next step draws anew
    return losses


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("graphs", 64), ("channels", 64), ("heads", 4), ("types", 10), ("steps", 20)):
        ap.add_argument(f"--{name}", type=int, default=value)
    a = ap.parse_args()
    for step, loss in enumerate(train(a.graphs, a.channels, a.heads, a.types, a.steps)):
        print(f"step {step:3d}  loss {loss:.5f}", flush=True)


if __name__ == "__main__":
    main()
