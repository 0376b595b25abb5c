"""GPU tests of the attention block's operators over the ranges of their sizes: fp32 inputs with a bf16 output, many heads, many
graphs, many irreps, parts that are longer than a run of sums, tensors of more than 2^31 values; and long graphs in columns of
wider tensors, captured into a graph, and beside rows of no graph.  Tolerances are those of test_gpu_attention."""
import numpy as np
import pytest

from gpu_cases import say
from test_gpu_attention import Case, at, offsets  # noqa: F401  (at: a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("qk,v,heads,lens,key_lens", [
    ("32x0e+32x1o", "64x0e", 4, (40, 33), None), ("96x0e", "100x0e", 1, (140, 99), None), ("7x0e+5x1o", "9x0e", 1, (1200,), None),
    ("256x0e", "256x0e+512x1o", 256, (23, 2), None), ("100x0e", "100x0e+100x1o", 100, (9, 1), (1400, 3)),
    ("+".join(f"{1 + l % 2}x{l % 4}{'eo'[l % 2]}" for l in range(16)), "4x0o+4x1e", 1, (33, 70), None)])
def test_types_heads_and_irreps(at, qk, v, heads, lens, key_lens):  # noqa: F811
    for i, (xb, yb) in enumerate(((False, True), (True, False), (True, True))):
        say(f"[case] ranges {qk} {v} heads={heads} {lens} {key_lens} x={'bf16' if xb else 'f32'} y={'bf16' if yb else 'f32'}")
        Case(qk, v, heads, lens, key_lens, xb, yb, cap=3.0 if i == 1 else 0.0, bias=i != 1, seed=40 + i).check(at)


@pytest.mark.parametrize("graphs", [64, 65, 4097, 9000])
@pytest.mark.parametrize("cross", [False, True])
def test_many_graphs(at, graphs, cross):  # noqa: F811
    """The search for a tile's graph in one to three steps, graphs without rows among them."""
    say(f"[case] {graphs} graphs cross={cross}")
    rng = np.random.default_rng(graphs)
    lens, keys = (tuple(int(n) for n in rng.integers(0, 4, graphs)) for _ in range(2))
    Case("4x0e", "4x0e", 1, lens, keys if cross else None, False, False, 0.0, True, 41).check(at)


@pytest.mark.parametrize("xb,yb", [(False, False), (True, True), (False, True)])
@pytest.mark.parametrize("lens,key_lens", [((300000,), (3,)), ((2,), (300000,)), ((1, 5), (280000, 9))])
def test_parts_longer_than_a_run(at, xb, yb, lens, key_lens):  # noqa: F811
    """64 parts of more than 4096 rows each, in either direction."""
    say(f"[case] long parts {lens} {key_lens} x={'bf16' if xb else 'f32'} y={'bf16' if yb else 'f32'}")
    Case("8x0e", "4x0e+1x1o", 1, lens, key_lens, xb, yb, 0.0, True, 42).check(at)


@pytest.mark.parametrize("xb", [False, True])
def test_a_long_graph_in_columns_and_beside_rows_of_no_graph(at, xb):  # noqa: F811
    """Runs' sums are kept in the rows of the results: strided ones, between columns and rows that stay as they were."""
    import torch

    say(f"[case] long graph in columns x={'bf16' if xb else 'f32'}")
    c = Case("8x0e+4x1o", "8x0e+4x1o", 2, (5000, 130), None, xb, False, 0.0, True, 43)
    ref_out, _, ref_saved, ref = c.run(at)
    h, n, f = c.layer(at), c.nq, 9
    rows = n + 2 * f
    wide = torch.full((rows, 65), float("nan"), dtype=c.q.dtype, device="cuda")
    gwide = torch.full((rows, 65), 7.0, device="cuda")
    cols = [slice(1 + 20 * i, 21 + 20 * i) for i in range(3)]
    for s, t in zip(cols, (c.q, c.k, c.v)):
        wide[f:f + n, s] = t
    grown = lambda t, fill: torch.cat([torch.full((f, t.shape[1]), fill, device="cuda"), t,  # noqa: E731
                                       torch.full((f, t.shape[1]), fill, device="cuda")])
    batch = at.Batch(rows, offsets(c.lens, f), grown(c.pos, float("nan")))
    out, gpos = (torch.full((rows, m), 7.0, device="cuda") for m in (20, 3))
    saved = torch.zeros(h.saved_size(rows), device="cuda")
    parts = [wide[:, s] for s in cols]
    at.tpconv_attention_forward(h, batch, *parts, slope=c.slope, out=out, saved=saved)
    gq, gk, gv = (gwide[:, s] for s in cols)
    got = at.tpconv_attention_backward(h, batch, *parts, out, saved, grown(c.g, float("nan")), slope=c.slope, want=("slope",),
                                       grad_q=gq, grad_k=gk, grad_v=gv, grad_pos=gpos)
    assert torch.equal(got[3], ref[3])
    for t, r in ((out, ref_out), (gq, ref[0]), (gk, ref[1]), (gv, ref[2]), (gpos, ref[4])):
        assert torch.equal(t[f:f + n], r) and torch.all(t[:f] == 7.0) and torch.all(t[f + n:] == 7.0)
    assert torch.all(gwide[:, 0] == 7.0) and torch.all(gwide[:, 61:] == 7.0)


@pytest.mark.parametrize("xb", [False, True])
def test_a_long_graph_captured(at, xb):  # noqa: F811
    """Forwards that save and that do not, and the backward, replayed with other inputs and eager work in between."""
    import torch

    say(f"[case] long graph captured x={'bf16' if xb else 'f32'}")
    c = Case("16x0e", "16x0e", 2, (4500, 40), None, xb, xb, 0.0, True, 44)
    h, b = c.layer(at), c.batch(at)
    saved = torch.empty(h.saved_size(c.nq), device="cuda")

    def step():
        plain = at.tpconv_attention_forward(h, b, c.q, c.k, c.v, slope=c.slope)
        out = at.tpconv_attention_forward(h, b, c.q, c.k, c.v, slope=c.slope, saved=saved)
        return (plain, out, *at.tpconv_attention_backward(h, b, c.q, c.k, c.v, out, saved, c.g, slope=c.slope,
                                                          want=c.want())[:5])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(4):
        for t in (c.q, c.k, c.v, c.g):
            t.copy_(torch.randn_like(t))
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in got]
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(kept, want)) and torch.equal(kept[0], kept[1])


# ---- tensors of more than 2^31 values ----------------------------------------------------

NODES, WIDE = 70000 * 32, 1024


@pytest.mark.parametrize("xb", [False, True])
def test_attention_past_32_bit_offsets(at, xb):  # noqa: F811
    """The last graphs of a batch whose tensors hold more than 2^31 values, as they are on their own."""
    import torch

    say(f"[case] attention past 2^31 values x={'bf16' if xb else 'f32'}")
    n, m = NODES, 96
    code = (at.TPCONV_F32, at.TPCONV_BF16)[xb]
    gen = torch.Generator("cuda").manual_seed(1)
    h = at.Attention(f"{WIDE}x0e", f"{WIDE}x0e", 16, x_dtype=code, y_dtype=code)
    q, k, v = (torch.zeros(n, WIDE, dtype=h.x_dtype, device="cuda") for _ in range(3))
    go, pos = torch.zeros(n, WIDE, device="cuda"), torch.randn(n, 3, device="cuda", generator=gen)
    slope = torch.rand(16, device="cuda", generator=gen)
    for t in (q, k, v, go):
        t[n - m:] = torch.randn(m, WIDE, device="cuda", generator=gen)

    def run(n, off, pos, q, k, v, go):
        b, saved = at.Batch(n, off, pos), torch.empty(h.saved_size(n), device="cuda")
        out = at.tpconv_attention_forward(h, b, q, k, v, slope=slope, saved=saved)
        got = at.tpconv_attention_backward(h, b, q, k, v, out, saved, go, slope=slope, want=("q", "k", "v", "pos"))
        return [t[n - m:].clone() for t in (out, *got) if t is not None]

    off = torch.arange(0, n + 1, 32, dtype=torch.int32, device="cuda")
    got = run(n, off, pos, q, k, v, go)
    small = [t[n - m:].clone() for t in (pos, q, k, v, go)]
    del q, k, v, go
    want = run(m, off[:4].clone(), *small)
    torch.cuda.synchronize()
    assert len(got) == 5 and all(torch.equal(a, b) for a, b in zip(got, want))
    torch.cuda.empty_cache()


def test_embedding_and_dropout_past_32_bit_offsets(at):  # noqa: F811
    import torch
    from oracle import attention as oa

    say("[case] embedding and dropout past 2^31 values")
    n, rows = NODES, 70
    gen = torch.Generator("cuda").manual_seed(2)
    z = torch.randint(0, rows, (n,), dtype=torch.int32, device="cuda", generator=gen)
    e, W = at.Embedding(rows, WIDE, 0.5), torch.randn(rows, WIDE, device="cuda", generator=gen)
    y = at.tpconv_embed_forward(e, z, W)
    assert torch.equal(y[-50:], 0.5 * W[z[-50:].long()])
    y.zero_()
    y[-1000:] = torch.randint(-8, 9, (1000, WIDE), device="cuda", generator=gen).float()  # sums that are exact
    gW = at.tpconv_embed_backward(e, z, y)
    assert torch.equal(gW, torch.zeros_like(W).index_add_(0, z[-1000:].long(), 0.5 * y[-1000:]))
    d, state = at.Dropout(f"{WIDE}x0e", 0.5), torch.tensor([5, 6], dtype=torch.int64, device="cuda")
    y.fill_(1.0)
    at.tpconv_dropout_forward(d, y, state, out=y)
    assert np.array_equal(y[-3:].double().cpu().numpy(), oa.dropout_factors(f"{WIDE}x0e", 3, 0.5, 5, 6, n - 3))
    del y
    torch.cuda.empty_cache()
