"""The attention block's operators together, as the example trains them: against the chained fp64 definitions, captured
into a graph, and several calls at once."""
import os
import sys

import numpy as np
import pytest

from gpu_cases import say
from oracle import attention as oa
from oracle import layers as ol

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def f64(t):
    return t.double().cpu().numpy()


def make(irreps, heads, types, sizes, seed):
    """(block, batch, node types, features, offsets) of a batch of graphs."""
    import torch
    import train_attention as ta
    from equivariant_gnn_tensor_receiver_amd import attention as at

    dev = torch.device("cuda:0")
    rng = np.random.default_rng(seed)
    n = sum(sizes)
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    to = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
    block = ta.Block(irreps, heads, types, 0.25, seed, dev)
    block.gamma = torch.rand(block.norm.num_weights, device=dev) + 0.5
    pos = to((2 * rng.standard_normal((n, 3))).astype(np.float32))
    index = to(rng.integers(0, types, n).astype(np.int32))
    x = to(rng.standard_normal((n, block.norm.features)).astype(np.float32))
    return block, at.Batch(n, to(off), pos), index, x, off


def test_example_runs():
    import train_attention

    say("[case] training steps of the attention example")
    losses = train_attention.train(graphs=12, channels=32, heads=4, types=5, steps=4)
    assert len(losses) == 5 and np.all(np.isfinite(losses))


@pytest.mark.parametrize("irreps,heads", [("16x0e", 2), ("8x0e+8x1o", 4), ("6x0e+4x1o+2x2e", 2)])
def test_block_against_the_chained_definitions(irreps, heads):
    """out and every gradient (features, weights, slopes, places, embedding).  Every operator is fp32-exact within the
    bounds of its own tests, each below 1e-4 of its largest value at these sizes; five of them in a row and their
    backward stay below 1e-3 of the results' largest values."""
    import torch
    from equivariant_gnn_tensor_receiver_amd import attention as at

    say(f"[case] block {irreps}")
    block, batch, index, x, off = make(irreps, heads, 7, (9, 1, 40, 17), 3)
    F = block.norm.features
    seed, offset = 11, 1 << 35
    state = torch.tensor([seed, offset], dtype=torch.int64, device="cuda")
    out = block.forward(x, batch, state)
    g = torch.randn_like(out)
    gx = block.backward(g)
    gE = at.tpconv_embed_backward(block.embed, index, gx)
    n = x.shape[0]
    one = np.zeros(n, dtype=np.int64)
    three = "+".join([irreps] * 3)
    y = ol.norm_forward(irreps, f64(x), f64(block.gamma), f64(block.beta))[0]
    qkv = ol.linear_forward(irreps, three, one, y, f64(block.P)).reshape(n, 3 * F)
    args = dict(offsets=off, scale=block.attention.scale, slope=f64(block.slope), pos=f64(batch.pos))
    q, k, v = qkv[:, :F], qkv[:, F:2 * F], qkv[:, 2 * F:]
    o = oa.attention(irreps, irreps, heads, q, k, v, **args)["out"]
    z = ol.linear_forward(irreps, irreps, one, o, f64(block.M)).reshape(n, F)
    mask = oa.dropout_factors(irreps, n, 0.25, seed, offset)
    ref = f64(x) + z * mask
    gz = f64(g) * mask
    go, gM = ol.linear_backward(irreps, irreps, one, o, f64(block.M), gz)
    a = oa.attention(irreps, irreps, heads, q, k, v, grad_out=np.asarray(go).reshape(n, F), **args)
    gqkv = np.concatenate([a["grad_q"], a["grad_k"], a["grad_v"]], 1)
    gy, gP = ol.linear_backward(irreps, three, one, y, f64(block.P), gqkv)
    rx, rg, rb = ol.norm_backward(irreps, f64(x), f64(block.gamma), np.asarray(gy).reshape(n, F))
    rx = np.asarray(rx).reshape(n, F) + f64(g)
    rE, _ = oa.embed_backward(index.cpu().numpy(), rx, 7, F ** 0.5)
    for name, got, want in (("out", out, ref), ("x", gx, rx), ("P", block.grad_p, gP), ("M", block.grad_m, gM),
                            ("gamma", block.grad_gamma, rg), ("beta", block.grad_beta, rb), ("E", gE, rE),
                            ("slope", block.grad_slope, a["grad_slope"]), ("pos", block.grad_pos, a["grad_pos"])):
        want = np.asarray(want)
        err = np.abs(f64(got).reshape(want.shape) - want).max()
        assert err <= 1e-3 * np.abs(want).max(), (name, err)


@pytest.mark.parametrize("sizes", [(9, 30, 17, 1), (1500,)])
def test_captured_and_replayed(sizes):
    """Forward and backward of everything in one graph, replayed with new inputs, new draws and eager work in between; the
    outputs equal the eager ones in every bit."""
    import torch
    from equivariant_gnn_tensor_receiver_amd import attention as at

    say(f"[case] captured {sizes}")
    block, batch, index, x, _ = make("8x0e+8x1o", 2, 5, sizes, 4)
    state = torch.tensor([3, 0], dtype=torch.int64, device="cuda")
    g = torch.randn_like(x)

    def step():
        e = at.tpconv_embed_forward(block.embed, index, block.E)
        out = block.forward(x + e, batch, state)
        gx = block.backward(g)
        gE = at.tpconv_embed_backward(block.embed, index, gx)
        return out, gx, gE, block.grad_p, block.grad_m, block.grad_slope, block.grad_pos, block.grad_gamma

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in range(4):
        x.copy_(torch.randn_like(x))
        index.copy_(torch.randint(0, 5, index.shape, dtype=torch.int32, device="cuda"))
        state[1] = 7 * i
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in got]
        want = step()
        torch.cuda.synchronize()
        for a, b in zip(kept, want):
            assert torch.equal(a, b)


def test_two_calls_at_once_on_two_streams():
    """One handle on two streams, each with a workspace of its own."""
    import torch
    from equivariant_gnn_tensor_receiver_amd import attention as at

    say("[case] two streams")
    h = at.Attention("32x0e", "32x0e", 1)
    off = torch.tensor([0, 1200], dtype=torch.int32, device="cuda")
    batch = at.Batch(1200, off)
    ts = [[torch.randn(1200, 32, device="cuda") for _ in range(4)] for _ in range(2)]

    def run(t, stream):
        saved = torch.empty(h.saved_size(1200), device="cuda")
        out = at.tpconv_attention_forward(h, batch, *t[:3], saved=saved, stream=stream)
        return (out, *at.tpconv_attention_backward(h, batch, *t[:3], out, saved, t[3], stream=stream)[:3])

    assert h.workspace_size(batch, at.OP_FORWARD) > 0
    want = [run(t, None) for t in ts]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ts]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        got = [run(t, s) for t, s in zip(ts, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_kernel_classes_are_timed():
    import torch
    from equivariant_gnn_tensor_receiver_amd import attention as at
    from equivariant_gnn_tensor_receiver_amd import tpconv as tp

    say("[case] kernel classes")
    block, batch, index, x, _ = make("8x0e", 2, 5, (20,), 5)
    L = at._lib()
    assert L.tpconv_kernel_timing(1) == 0
    try:
        block.forward(at.tpconv_embed_forward(block.embed, index, block.E), batch,
                      torch.zeros(2, dtype=torch.int64, device="cuda"))
        times = {}
        import ctypes

        for name in ("attention", "embed", "dropout"):
            n, ms = ctypes.c_int64(), ctypes.c_double()
            assert L.tpconv_kernel_timing_read(tp.KERNELS.index(name), ctypes.byref(n), ctypes.byref(ms)) == 0
            times[name] = n.value
    finally:
        L.tpconv_kernel_timing(0)
    assert times == dict(attention=1, embed=1, dropout=1)
