"""Trains one interaction block on synthetic data: layer norm -> streaming convolution -> linear layer per element.

    x --norm--> y --conv(graph, W)--> z --linear(element, V)--> out,   loss = mean((out - target)^2) / 2

The target is the same block with other weights.  The gradients run back through the three layers, and both weight
banks (W[K][P][C_in][C_out] of the convolution, V[elements][...] of the linear layer) take orthogonalised (Muon)
steps; the norm's weights and biases, which are vectors, take plain gradient steps.

    python examples/train_block.py [--nodes 512] [--channels 32] [--lmax 2] [--elements 5] [--steps 20]
"""
from __future__ import annotations

import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from equivariant_gnn_tensor_receiver_amd import inputs, layers  # noqa: E402
from equivariant_gnn_tensor_receiver_amd import tpconv as tp  # noqa: E402


class Block:
    """The layers, their plans and workspaces, and the weights."""

    def __init__(self, irreps, lmax, num_basis, elements, graph, pos, seed, device):
        self.plan = tp.Plan(irreps, irreps, lmax, num_basis)
        self.graph, self.pos = tp.tpconv_graph_prepare(self.plan, graph), pos
        self.norm = layers.Norm(irreps)
        self.linear = layers.Linear(irreps, irreps, elements)
        gen = torch.Generator(device).manual_seed(seed)
        fan = self.plan.ch_in
        self.W = torch.randn(self.plan.w_shape, generator=gen, device=device) * (num_basis * fan) ** -0.5
        self.V = torch.randn(self.linear.w_shape, generator=gen, device=device) * fan ** -0.5
        self.gamma = torch.ones(self.norm.num_weights, device=device)
        self.beta = torch.zeros(self.norm.num_biases, device=device)
        # optimiser: one handle per weight bank and its momentum
        self.opt_w, self.opt_v = (layers.Muon(layers.weight_blocks(v)) for v in (self.plan, self.linear))
        self.mom_w, self.mom_v = torch.zeros_like(self.W), torch.zeros_like(self.V)

    def forward(self, x, groups):
        n = x.shape[0]
        self.stats = torch.empty(self.norm.stats_shape(n), device=x.device)
        self.y = layers.tpconv_norm_forward(self.norm, x, self.gamma, self.beta, stats=self.stats)
        self.z = tp.tpconv_forward(self.plan, self.graph, self.pos, self.y, self.W)
        return layers.tpconv_linear_forward(self.linear, groups, self.z, self.V)

    def backward(self, x, groups, grad_out):
        """The gradient of x; the weights' gradients stay in the block."""
        grad_z, self.grad_v = layers.tpconv_linear_backward(self.linear, groups, self.z, self.V, grad_out)
        grad_y, self.grad_w, _ = tp.tpconv_backward(self.plan, self.graph, self.pos, self.y, self.W, grad_z,
                                                    want=("x", "W"))
        grad_x, self.grad_gamma, self.grad_beta = layers.tpconv_norm_backward(self.norm, x, self.gamma, grad_y,
                                                                              stats=self.stats)
        return grad_x

    def update(self, lr):
        for opt, w, g, m in ((self.opt_w, self.W, self.grad_w, self.mom_w),
                             (self.opt_v, self.V, self.grad_v, self.mom_v)):
            layers.tpconv_muon_step(opt, w, g, m, lr, W_out=w, momentum_out=m)
        self.gamma -= lr * self.grad_gamma
        self.beta -= lr * self.grad_beta


def train(nodes=512, channels=32, lmax=2, elements=5, degree=12, steps=20, lr=0.02, seed=0, device="cuda:0"):
    """The loss before every step, and after the last."""
    device = torch.device(device)
    irreps = "+".join(f"{channels}x{l}{'eo'[l % 2]}" for l in range(lmax + 1))
    pos, rowptr, senders, rng = inputs.random_graph(nodes, degree, seed)
    to = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(device)
    graph, pos = tp.Graph(to(rowptr), to(senders)), to(pos)
    block, teacher = (Block(irreps, lmax, 8, elements, graph, pos, s, device) for s in (seed, seed + 1))
    x = torch.randn(block.plan.in_shape(nodes), generator=torch.Generator(device).manual_seed(seed), device=device)
    groups = layers.tpconv_linear_groups(block.linear, to(rng.integers(0, elements, nodes).astype(np.int32)))
    target = teacher.forward(x, groups)
    losses = []
    for step in range(steps + 1):
        diff = block.forward(x, groups) - target
        losses.append(float(diff.square().mean()) / 2)
        if step == steps:
            break
        block.backward(x, groups, diff / diff.numel())
        block.update(lr)
    return losses


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("nodes", 512), ("channels", 32), ("lmax", 2), ("elements", 5), ("steps", 20)):
        ap.add_argument(f"--{name}", type=int, default=value)
    a = ap.parse_args()
    for step, loss in enumerate(train(a.nodes, a.channels, a.lmax, a.elements, steps=a.steps)):
        print(f"step {step:3d}  loss {loss:.5f}", flush=True)


if __name__ == "__main__":
    main()
