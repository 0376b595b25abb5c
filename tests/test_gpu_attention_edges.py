"""GPU tests of the attention at the edges of its arguments: forwards that save and that do not, scales of zero and below,
values that are not finite in launches cut into parts, long graphs among many small ones, offsets that decrease.  Tolerances
not derived here are those of test_gpu_attention."""
import numpy as np
import pytest

from gpu_cases import say
from test_gpu_attention import Case, U, at, cuda, f64, near, offsets  # noqa: F401  (at: a fixture)

pytestmark = pytest.mark.gpu


# ---- forwards that save and that do not ---------------------------------------------


@pytest.mark.parametrize("qk,v,heads", [("32x0e", "32x0e", 1), ("64x0e+32x1o", "64x0e+32x1o", 8), ("100x0e", "128x0e", 1),
                                        ("200x0e", "256x0e", 1), ("7x0e+5x1o", "3x0e+31x1o", 1)])
@pytest.mark.parametrize("lens,key_lens", [((5, 0, 33, 1), None), ((1200,), None), ((400, 200, 100), None),
                                           ((1, 2), (700, 900)), ((40,), (9000,))])
def test_a_bf16_forward_is_the_same_whether_it_saves_or_not(at, qk, v, heads, lens, key_lens):  # noqa: F811
    """One result of one set of inputs: the weights enter the sums with the same bits either way."""
    import torch

    for cap, bias in ((0.0, True), (4.0, False), (0.0, False)):
        say(f"[case] saving or not {qk} {v} {lens} {key_lens} cap={cap} bias={bias}")
        c = Case(qk, v, heads, lens, key_lens, True, True, cap, bias, 31)
        h, b = c.layer(at), c.batch(at)
        saved = torch.empty(h.saved_size(c.nq), device="cuda")
        out = at.tpconv_attention_forward(h, b, c.q, c.k, c.v, slope=c.slope, saved=saved)
        assert torch.equal(out, at.tpconv_attention_forward(h, b, c.q, c.k, c.v, slope=c.slope))
        # the saved fp32 output is the one that was rounded
        assert torch.equal(out, saved[2 * heads * c.nq:].view(c.nq, -1).bfloat16())

# ---- scales of zero and below ---------------------------------------------------------

SCALED = [("8x0e", "8x0e", 2), ("66x0e", "62x0e", 2), ("32x0e+32x1o+32x2e", "32x0e+32x1o+32x2e", 2), ("100x0e", "128x0e", 1)]


class Negated(Case):
    """The scores of a case from its queries with the other sign and its scale with the other sign."""

    def run(self, at, **kw):  # noqa: F811
        self.scale, self.q = -self.scale, -self.q
        out, plain, saved, grads = super().run(at, **kw)
        self.scale, self.q = -self.scale, -self.q
        return out, plain, saved, (-grads[0], *grads[1:])


@pytest.mark.parametrize("qk,v,heads", SCALED)
@pytest.mark.parametrize("xb", [False, True])
@pytest.mark.parametrize("lens,key_lens", [((1,), None), ((33, 65), None), ((130, 3), None), ((1111,), None),
                                           ((2, 1), (700, 31))])
def test_scales_of_zero(at, qk, v, heads, xb, lens, key_lens):  # noqa: F811
    """All keys weigh the same (or by their distance alone); rows of a tile that are not there weigh nothing."""
    for cap, bias in ((0.0, False), (0.0, True), (4.0, False)):
        for scale in (0.0, 1e-42):
            say(f"[case] scale {scale} {qk} {v} {lens} {key_lens} x={'bf16' if xb else 'f32'} cap={cap} bias={bias}")
            c = Case(qk, v, heads, lens, key_lens, xb, xb, cap, bias, 32)
            c.scale = scale
            c.check(at)


@pytest.mark.parametrize("qk,v,heads", SCALED)
@pytest.mark.parametrize("xb", [False, True])
@pytest.mark.parametrize("lens,key_lens", [((33, 65), None), ((130, 3), None), ((1111,), None), ((2, 1), (700, 31))])
def test_scales_below_zero(at, qk, v, heads, xb, lens, key_lens):  # noqa: F811
    for cap, bias in ((0.0, False), (0.0, True), (4.0, False)):
        say(f"[case] negated {qk} {v} {lens} {key_lens} x={'bf16' if xb else 'f32'} cap={cap} bias={bias}")
        Negated(qk, v, heads, lens, key_lens, xb, xb, cap, bias, 33).check(at)

# ---- values that are not finite -----------------------------------------------------------


@pytest.mark.parametrize("xb", [False, True])
def test_a_nan_under_a_weight_of_zero_shows_whether_the_launch_is_cut_into_parts_or_not(at, xb):  # noqa: F811
    """Two keys' worth of scores, 300 apart: the low half of the keys has weights that vanish, 0 * NaN is NaN all the same."""
    import torch

    for graphs in (1, 1000):  # a few blocks, cut into parts; enough blocks without
        say(f"[case] NaN under a weight of zero graphs={graphs} x={'bf16' if xb else 'f32'}")
        n = 2560
        h = at.Attention("8x0e", "8x0e", 1, 1.0, 0.0, at.TPCONV_BF16 if xb else at.TPCONV_F32)
        off, key_off = offsets((1,) * graphs), offsets((n,) + (1,) * (graphs - 1))
        b = at.Batch(graphs, off, None, n + graphs - 1, key_off)
        assert (h.workspace_size(b, at.OP_FORWARD) > 0) == (graphs == 1)
        q, k, v = (cuda(np.ones((m, 8)), xb) for m in (graphs, n + graphs - 1, n + graphs - 1))
        k[:] = 0
        k[n // 2:n, 0] = 300.0
        v[7, 3] = float("nan")
        out = at.tpconv_attention_forward(h, b, q, k, v)
        assert out[0, 3].isnan()
        # the others are a sum times 1 / l, which is rounded, as each of the at most 64 parts' products is: 65 U off, not 0
        out[0, 3] = 1.0
        assert torch.all((out - 1.0).abs() <= 65 * U)

# ---- long graphs among many small ones ------------------------------------------------------

LONG, GRAPHS = 40000, 128


@pytest.mark.parametrize("xb", [False, True])
def test_sums_of_a_long_graph_among_small_ones(at, xb):  # noqa: F811
    """Equal weights over LONG keys.  fp32: values 1 + 2^-16, whose second pieces the matrix instructions add eight at a time
    (2^-13): exact while the sum is below 2^11, and lost beside it from there on, half a unit in its last place or less.  A run
    of 4096 keys loses 2^-16 (4096 - 2^11) / 4096 = 2^-17 of itself at most; one run over the graph would lose 2^-16 (LONG -
    2^11) / LONG = 1.45e-5, twice as much as is allowed.  bf16: every other value 2^-14 in place of one, eight at a time 4 +
    2^-12: exact below 2^12, which a run's sum of 2^11 does not reach; one run over the graph would lose 4.8e-5.  The runs'
    sums, the division and the product are rounded: LONG / 4096 + 2 roundings, relative to a mean of terms of one sign."""
    import torch

    say(f"[case] long graph forward x={'bf16' if xb else 'f32'}")
    n = LONG + 30 * (GRAPHS - 1)
    row = np.full(n, 1 + 2.0 ** -16) if not xb else np.where(np.arange(n) % 2 == 0, 1.0, 2.0 ** -14)
    v = cuda(np.repeat(row[:, None], 64, 1), xb)
    assert np.all(f64(v[:, 0]) == row)  # exact in its type
    code = (at.TPCONV_F32, at.TPCONV_BF16)[xb]
    h = at.Attention("64x0e", "64x0e", 8, 1.0, 0.0, code, code)
    b = at.Batch(GRAPHS, offsets((1,) * GRAPHS), None, n, offsets((LONG,) + (30,) * (GRAPHS - 1)))
    q, k = torch.zeros_like(v[:GRAPHS]), torch.randn(n, 64, device="cuda").to(v.dtype)
    saved = torch.empty(h.saved_size(GRAPHS), device="cuda")
    out = at.tpconv_attention_forward(h, b, q, k, v, saved=saved)
    got = f64(saved[2 * 8 * GRAPHS:].view(GRAPHS, 64)[0] if xb else out[0])
    mean = row[:LONG].mean()
    lost = 0.0 if xb else 2.0 ** -17
    assert np.all(np.abs(got - mean) <= (lost + (LONG / 4096 + 2) * U) * mean), np.abs(got / mean - 1).max()
    assert torch.equal(out, at.tpconv_attention_forward(h, b, q, k, v))


@pytest.mark.parametrize("xb", [False, True])
def test_gradient_sums_of_a_long_graph_among_small_ones(at, xb):  # noqa: F811
    """The same with LONG queries of one key each: the gradient of its value is the sum of their grad_out, 1 + 2^-16, in
    three pieces whatever the inputs' type."""
    import torch

    say(f"[case] long graph gradient x={'bf16' if xb else 'f32'}")
    n = LONG + 30 * (GRAPHS - 1)
    code = (at.TPCONV_F32, at.TPCONV_BF16)[xb]
    h = at.Attention("64x0e", "64x0e", 8, 1.0, 0.0, code, code)
    b = at.Batch(n, offsets((LONG,) + (30,) * (GRAPHS - 1)), None, GRAPHS, offsets((1,) * GRAPHS))
    q, k = (torch.randn(m, 64, device="cuda").to((torch.float32, torch.bfloat16)[xb]) for m in (n, GRAPHS))
    saved = torch.empty(h.saved_size(n), device="cuda")
    out = at.tpconv_attention_forward(h, b, q, k, k, saved=saved)
    go = torch.full((n, 64), 1 + 2.0 ** -16, device="cuda")
    _, _, gv, *_ = at.tpconv_attention_backward(h, b, q, k, k, out, saved, go, want=("v",))
    want = LONG * (1 + 2.0 ** -16)
    allowed = (2.0 ** -17 + (LONG / 4096 + 2) * U) * want
    assert np.all(np.abs(f64(gv[0]) - want) <= allowed), np.abs(f64(gv[0]) / want - 1).max()


@pytest.mark.parametrize("qk,v,heads", [("16x0e", "8x0e+8x1o", 2), ("5x0e+2x1o", "3x0e+2x1o", 1), ("160x0e", "100x0e", 1)])
@pytest.mark.parametrize("xb,yb", [(False, False), (True, True)])
@pytest.mark.parametrize("cap,bias", [(0.0, True), (3.0, False)])
def test_several_runs_of_rows(at, qk, v, heads, xb, yb, cap, bias):  # noqa: F811
    """Graphs longer than one run, in whole runs and beyond: references that move from run to run, sums kept in the results."""
    for lens, key_lens in (((4500, 7), None), ((3, 40), (8192, 9)), ((4097, 1), (33, 2))):
        say(f"[case] runs {qk} {v} {lens} {key_lens} x={'bf16' if xb else 'f32'} cap={cap} bias={bias}")
        Case(qk, v, heads, lens, key_lens, xb, yb, cap, bias, 34).check(at)


@pytest.mark.parametrize("xb", [False, True])
def test_scores_that_grow_from_run_to_run(at, xb):  # noqa: F811
    """The largest score of each run far above those before, and far below: keys times 1, 20, 3 and 60."""
    import torch

    say(f"[case] growing scores x={'bf16' if xb else 'f32'}")
    c = Case("16x0e", "16x0e", 1, (40, 900), (13000, 5), xb, xb, 0.0, False, 35)
    for run in range(4):
        c.k[4096 * run:4096 * (run + 1)] *= (1, 20, 3, 60)[run]
    c.check(at)

# ---- offsets that decrease or leave the rows ------------------------------------------------


class Guarded:
    """Tensors between margins of marks, which no kernel may touch."""

    def __init__(self):
        self.made = []

    def __call__(self, shape, fill=0.0, dtype=None, margin=4096):
        import torch

        dtype = dtype or torch.float32
        n = int(np.prod(shape))
        whole = torch.full((n + 2 * margin,), 77, dtype=dtype, device="cuda")
        t = whole[margin:margin + n].view(shape)
        t.fill_(fill)
        self.made.append((whole, margin, n))
        return t

    def check(self):
        for whole, margin, n in self.made:
            assert bool((whole[:margin] == 77).all()) and bool((whole[margin + n:] == 77).all())


BAD = [[0, 50, 20, 64], [-5, 10, 1000, 2000], [64, 0, 64, 0], [2 ** 31 - 1, -2 ** 31, 5, 64], [64, 64, 0, 0], [3, 3, 3, 3]]


@pytest.mark.parametrize("xb", [False, True])
@pytest.mark.parametrize("n,heads", [(64, 2), (700, 1)])  # whole, and cut into parts both ways
@pytest.mark.parametrize("bias", [False, True])
def test_bad_offsets_write_inside_their_tensors(at, xb, n, heads, bias):  # noqa: F811
    """Outputs, saved values, every gradient and a workspace of just the size that is needed keep their margins; self form and
    cross form, offsets of the queries, of the keys, and of both."""
    import torch

    code = (at.TPCONV_F32, at.TPCONV_BF16)[xb]
    h = at.Attention("8x0e", "8x0e", heads, 0.3, 0.0, code, code)
    good = [0, n // 3, n // 2, n]
    for bad in BAD:
        bad = [v * (n // 64) if 0 <= v <= 64 else v for v in bad]
        for mine, keys in ((bad, None), (bad, good), (good, bad), (bad, bad)):
            say(f"[case] bad offsets {mine} {keys} n={n} x={'bf16' if xb else 'f32'} bias={bias}")
            g = Guarded()
            off = [None if o is None else torch.tensor(o, dtype=torch.int64).to(torch.int32).cuda() for o in (mine, keys)]
            x = [cuda(np.random.default_rng(i).standard_normal((n, 8)), xb) for i in range(3)]
            pos = cuda(np.random.default_rng(3).standard_normal((n, 3))) if bias else None
            slope = torch.full((heads,), 0.5, device="cuda") if bias else None
            batch = at.Batch(n, off[0], pos, *(() if keys is None else (n, off[1], pos)))
            out, saved = g((n, 8), dtype=x[0].dtype), g((h.saved_size(n),))
            size = lambda op: g((h.workspace_size(batch, op),), 0, torch.uint8)  # noqa: E731
            at.tpconv_attention_forward(h, batch, *x, slope=slope, out=out, saved=saved, workspace=size(at.OP_FORWARD))
            at.tpconv_attention_forward(h, batch, *x, slope=slope, out=out, workspace=size(at.OP_FORWARD))
            grads = dict(grad_q=g((n, 8)), grad_k=g((n, 8)), grad_v=g((n, 8)))
            if bias:
                grads.update(grad_slope=g((heads,)), grad_pos=g((n, 3)))
                if keys is not None:
                    grads["grad_key_pos"] = g((n, 3))
            at.tpconv_attention_backward(h, batch, *x, out, saved, g((n, 8), 1.0), slope=slope, want=(),
                                         workspace=size(at.OP_BACKWARD), **grads)
            torch.cuda.synchronize()
            g.check()


# ---- padded batches ---------------------------------------------------------------------------


def test_a_padded_batch_with_cleared_results_through_the_next_layer(at):  # noqa: F811
    """Rows behind the last graph: NaN in the inputs, zeros in the results that the caller made; the next layer runs over all
    rows.  Its weight gradient is a sum of products within 2^-21 of theirs over 3 rows of N nodes, added in fp32."""
    import torch
    from equivariant_gnn_tensor_receiver_amd import layers
    from oracle import layers as ol

    say("[case] padded batch")
    irreps, pad = "8x0e+8x1o", 61
    c = Case(irreps, irreps, 2, (7, 40), bias=True, seed=36)
    n, whole = c.nq, c.nq + pad
    grown = lambda t, fill: torch.cat([t, torch.full((pad, t.shape[1]), fill, device="cuda")])  # noqa: E731
    nan = float("nan")
    q, k, v, pos, g = (grown(t, nan) for t in (c.q, c.k, c.v, c.pos, c.g))
    h, batch = c.layer(at), at.Batch(whole, offsets(c.lens), pos)
    zeros = lambda f: torch.zeros(whole, f, device="cuda")  # noqa: E731
    saved = torch.empty(h.saved_size(whole), device="cuda")
    out = at.tpconv_attention_forward(h, batch, q, k, v, slope=c.slope, out=zeros(32), saved=saved)
    grads = at.tpconv_attention_backward(h, batch, q, k, v, out, saved, g, slope=c.slope, want=("slope",), grad_q=zeros(32),
                                         grad_k=zeros(32), grad_v=zeros(32), grad_pos=zeros(3))
    ref_out, _, _, ref = c.run(at)
    for t, r in ((out, ref_out), *zip((*grads[:3], grads[4]), (*ref[:3], ref[4]))):
        assert torch.equal(t[:n], r) and torch.all(t[n:] == 0)
    assert torch.equal(grads[3], ref[3])
    lin = layers.Linear(irreps, irreps, 1)
    W = torch.randn(lin.w_shape, device="cuda")
    _, gW = layers.tpconv_linear_backward(lin, layers.Groups(whole), out, W, grown(c.g, 1.0))
    one = np.zeros(n, dtype=np.int64)
    want = np.asarray(ol.linear_backward(irreps, irreps, one, f64(ref_out), f64(W), f64(c.g))[1])
    mag = np.asarray(ol.linear_backward(irreps, irreps, one, np.abs(f64(ref_out)), np.abs(f64(W)), np.abs(f64(c.g)))[1])
    near(gW.reshape(want.shape), want, (2.0 ** -21 + 3 * n * U) * mag, "weight gradient")
