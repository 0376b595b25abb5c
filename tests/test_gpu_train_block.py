"""The node layers and the convolution together, as the example trains them, and the whole block's gradients."""
import os
import sys

import numpy as np
import pytest

from gpu_cases import say

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_training_lowers_the_loss():
    import train_block

    say("[case] twelve training steps of the block")
    losses = train_block.train(nodes=200, channels=16, lmax=1, elements=3, steps=12)
    assert np.all(np.isfinite(losses)) and losses[-1] < 0.5 * losses[0]


def test_block_gradient_against_the_oracles():
    """dL/dx, dL/dgamma, dL/dbeta, dL/dW and dL/dV through the three layers against the fp64 definitions chained."""
    import torch
    import train_block
    from equivariant_gnn_tensor_receiver_amd import inputs
    from equivariant_gnn_tensor_receiver_amd import layers as ly
    from equivariant_gnn_tensor_receiver_amd import tpconv as tp
    from oracle import layers as ol
    from oracle import tpconv as otp

    say("[case] gradients of the block against the chained definitions")
    ir, N, G = "8x0e+8x1o", 40, 3
    pos, rowptr, senders, rng = inputs.random_graph(N, 10, 3)
    dev = torch.device("cuda:0")
    to = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)
    b = train_block.Block(ir, 1, 8, G, tp.Graph(to(rowptr), to(senders)), to(pos), 5, dev)
    b.gamma = torch.rand(b.norm.num_weights, device=dev) + 0.5
    x = torch.randn(b.plan.in_shape(N), device=dev)
    group = rng.integers(0, G, N).astype(np.int32)
    groups = ly.tpconv_linear_groups(b.linear, to(group))
    out = b.forward(x, groups)
    g = torch.randn_like(out)
    gx = b.backward(x, groups, g)
    f = lambda t: t.double().cpu().numpy()
    prob = otp.Problem(ir, ir, 1, 8)
    rcv = otp.csr_receivers(rowptr)
    shape = (N, prob.D_in, prob.C_in)
    y = ol.norm_forward(ir, f(x), f(b.gamma), f(b.beta))[0].reshape(shape)
    z = otp.forward(prob, pos, senders, rcv, y, f(b.W))
    ref = ol.linear_forward(ir, ir, group, z, f(b.V))
    gz, gV = ol.linear_backward(ir, ir, group, z, f(b.V), f(g))
    gy, gW, _ = otp.backward(prob, pos, senders, rcv, y, f(b.W), gz.reshape(z.shape))
    rx, rg, rb = ol.norm_backward(ir, f(x), f(b.gamma), gy)
    # the convolution's own bounds (1e-4 forward, 1e-3 gradients) carry over: the layers around it are fp32-exact
    for got, want, tol in ((out, ref, 1e-4), (gx, rx, 1e-3), (b.grad_v, gV, 1e-3), (b.grad_w, gW, 1e-3),
                           (b.grad_gamma, rg, 1e-3), (b.grad_beta, rb, 1e-3)):
        want = np.asarray(want)
        assert np.abs(f(got).reshape(want.shape) - want).max() <= tol * np.abs(want).max()
