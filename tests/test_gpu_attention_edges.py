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
