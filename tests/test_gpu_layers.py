"""GPU parity of the node layers with their fp64 definitions.

Tolerances, fixed before the first run (u = 2^-24, the rounding of fp32):
  norm:    a value passes about sixteen roundings on top of its block's sums, whose error grows with the mean over
           the deviation: 64 u (1 + |mu| / sigma) of the largest value; parameter gradients 256 u of the sum of their
           terms' magnitudes (runs of a few hundred terms); bf16 results half a unit in the last place of their
           8-bit significand more.
  linear:  per element, of the sum S of its terms' magnitudes: one rounding per 16-long product and piece,
           (6 K / 16 + 16) u, and 2^-21 for the pieces left out.
  muon:    a rounding of step t grows by at most the later steps' slopes (at most a = 3.4445 each): five steps pass on
           3.4445^5 = 485 times 2^-21 (operands of 22 bits, three products) of the Frobenius norm of X, which starts
           at 1, from each step: 5 * 485 * 2^-21 = 1.2e-3 absolute in the Frobenius norm; one step 4 * 2^-21.
"""
import numpy as np
import pytest

from gpu_cases import say
from oracle import layers as ol

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def ly():
    from equivariant_gnn_tensor_receiver_amd import layers

    return layers


def cuda(a, bf16=False):
    import torch

    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda()
    return t.bfloat16() if bf16 else t


def f64(t):
    return t.double().cpu().numpy()


def half_ulp(a):
    """Half a unit in the last place of a's values in bf16 (8-bit significand: 2^-8 of the power of two below)."""
    a = np.abs(a)
    return np.where(a > 0, 2.0 ** (np.floor(np.log2(np.where(a > 0, a, 1.0))) - 8), 0.0)


def misaligned(t):
    """The same values one element past an aligned address."""
    import torch

    s = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)[1:]
    s.copy_(t.reshape(-1))
    return s.view(t.shape)


# ---- layer norm ---------------------------------------------------------------------

NORM_IRREPS = ["1x0e", "3x0e", "8x0e+8x1o", "5x0e+3x1o+2x1e+4x0o+1x3o", "32x0e+32x1o+32x2e", "64x0e+64x1o+64x2e+64x3o",
               "128x0e+130x1o+127x2e", "255x0e+300x1o", "1031x0e", "4096x0e", "2048x0e+1024x1o", "8200x0e+12x2e",
               "20000x0e"]


def norm_data(irreps, N, seed, shift=0.0):
    rng = np.random.default_rng(seed)
    F = ol.irreps(irreps)[1]
    x = (rng.standard_normal((N, F)) * (0.1 + rng.random((N, 1))) + shift).astype(np.float32)
    blocks = ol.irreps(irreps)[0]
    nw, nb = sum(b[0] for b in blocks), sum(b[0] for b in blocks if b[2] == "0e")
    return (x, rng.standard_normal(nw).astype(np.float32), rng.standard_normal(nb).astype(np.float32),
            rng.standard_normal((N, F)).astype(np.float32))


def check_norm(ly, irreps, x, w, b, g, xb=False, yb=False, align=True, eps=1e-5):
    """Forward, statistics and backward of one case (x: what the GPU gets, exact in its type)."""
    import torch

    norm = ly.Norm(irreps, eps, ly.TPCONV_BF16 if xb else ly.TPCONV_F32, ly.TPCONV_BF16 if yb else ly.TPCONV_F32)
    X, Wt, B, G = cuda(x, xb), cuda(w), cuda(b), cuda(g)
    if not align:
        X, G = misaligned(X), misaligned(G)
    x = f64(X)
    N = x.shape[0]
    stats = torch.full(norm.stats_shape(N), float("nan"), device="cuda")
    y = ly.tpconv_norm_forward(norm, X, Wt, B, stats=stats)
    gx, gw, gb = ly.tpconv_norm_backward(norm, X, Wt, G, stats=stats)
    gx2, gw2, gb2 = ly.tpconv_norm_backward(norm, X, Wt, G)
    torch.cuda.synchronize()
    ry, rs = ol.norm_forward(irreps, x, w, b, eps)
    rgx, rgw, rgb = ol.norm_backward(irreps, x, w, g, eps)
    spread = 1.0 + np.abs(rs[..., 0] * rs[..., 1]).max(initial=0.0)
    tol = 64 * U * spread
    near = tol * np.abs(ry).max(initial=0.0)
    # (a value that fp32 errors carry over a power of two rounds in the next binade)
    assert np.all(np.abs(f64(y) - ry) <= near + (half_ulp(np.abs(ry) + near) if yb else 0.0))
    assert np.abs(f64(stats)[..., 1] / rs[..., 1] - 1).max(initial=0.0) <= tol
    assert np.abs(f64(stats)[..., 0] - rs[..., 0]).max(initial=0.0) <= 64 * U * np.abs(x).max(initial=0.0)
    # magnitudes of the parameter gradients' terms
    one = np.ones(len(w))
    z, _ = ol.norm_forward(irreps, x, one, None, eps)
    at = 0
    for mul, n, kind, off in ol.irreps(irreps)[0]:
        t = np.abs(z[:, off:off + n * mul] * g[:, off:off + n * mul]).sum(0).reshape(n, mul).sum(0)
        for v in (gw, gw2):
            assert np.all(np.abs(f64(v)[at:at + mul] - rgw[at:at + mul]) <= (256 * U + tol) * t.max(initial=0.0) + 1e-30)
        at += mul
    for v in (gb, gb2):
        assert np.abs(f64(v) - rgb).max(initial=0.0) <= 256 * U * np.abs(g).sum(0).max(initial=0.0)
    scale = max(np.abs(rgx).max(initial=0.0), (np.abs(w).max() * np.abs(g).max(initial=0.0) * rs[..., 1].max(initial=0.0)))
    for v in (gx, gx2):
        assert np.abs(f64(v) - rgx).max(initial=0.0) <= tol * scale
    return y, gx, gw, gb


@pytest.mark.parametrize("irreps", NORM_IRREPS)
@pytest.mark.parametrize("xb,yb", [(False, False), (True, True), (False, True), (True, False)])
def test_norm_matches_definition(ly, irreps, xb, yb):
    for N in (1, 3, 61) if len(irreps) < 16 else (5,):
        say(f"[case] norm {irreps} N={N} x={'bf16' if xb else 'f32'} y={'bf16' if yb else 'f32'}")
        check_norm(ly, irreps, *norm_data(irreps, N, N), xb=xb, yb=yb)


@pytest.mark.parametrize("irreps,N", [("32x0e+32x1o+32x2e", 3001), ("7x0e+5x1o", 2999), ("1000x0e", 1500)])
def test_norm_many_nodes(ly, irreps, N):
    say(f"[case] norm {irreps} N={N}")
    check_norm(ly, irreps, *norm_data(irreps, N, 3))
    check_norm(ly, irreps, *norm_data(irreps, N, 4), align=False)


def test_norm_large_mean_keeps_the_variance(ly):
    say("[case] norm with a mean of 300 deviations")
    check_norm(ly, "64x0e+8x1o", *norm_data("64x0e+8x1o", 33, 5, shift=300.0))
    check_norm(ly, "1500x0e", *norm_data("1500x0e", 9, 6, shift=300.0))


def test_norm_degenerate_rows(ly):
    """Zero rows and constant rows have no deviation; a row that is not finite stays in its own row."""
    import torch

    for irreps in ("8x0e+4x1o", "700x0e+300x1o"):
        say(f"[case] degenerate rows of {irreps}")
        x, w, b, g = norm_data(irreps, 6, 7)
        x[1] = 0.0
        x[2] = 0.75  # exact sums: the deviation of the scalars is exactly zero
        check_norm(ly, irreps, x, w, b, g)
        norm = ly.Norm(irreps)
        good = ly.tpconv_norm_forward(norm, cuda(x), cuda(w), cuda(b))
        assert torch.equal(good[1][:len(b)], cuda(b))
        x[4, 1] = np.nan
        x[5, 0] = np.inf
        y = ly.tpconv_norm_forward(norm, cuda(x), cuda(w), cuda(b))
        gx, _, _ = ly.tpconv_norm_backward(norm, cuda(x), cuda(w), cuda(g))
        assert torch.equal(y[:4], good[:4]) and torch.isnan(y[4, :len(b)]).all() and torch.isnan(y[5, 0])
        assert torch.isfinite(gx[:4]).all()


def test_norm_without_parameters_and_single_gradients(ly):
    import torch

    say("[case] norm without weight and bias, wanted gradients one at a time")
    irreps = "12x0e+5x1o"
    x, w, b, g = norm_data(irreps, 17, 8)
    norm = ly.Norm(irreps)
    X, G = cuda(x), cuda(g)
    y = ly.tpconv_norm_forward(norm, X)
    assert np.abs(f64(y) - ol.norm_forward(irreps, x)[0]).max() <= 64 * U * 4 * np.abs(f64(y)).max()
    full = ly.tpconv_norm_backward(norm, X, None, G)
    assert np.abs(f64(full[0]) - ol.norm_backward(irreps, x, None, g)[0]).max() <= 64 * U * 4 * np.abs(f64(full[0])).max()
    for i, name in enumerate(("x", "weight", "bias")):
        one = ly.tpconv_norm_backward(norm, X, None, G, want=(name,))
        assert [v is None for v in one] == [k != i for k in range(3)] and torch.equal(one[i], full[i])
    # no 0e block: an empty bias gradient; no nodes: zero gradients
    odd = ly.Norm("4x1o")
    assert ly.tpconv_norm_backward(odd, X[:2, :12].contiguous(), None, G[:2, :12].contiguous())[2].numel() == 0
    gx, gw, gb = ly.tpconv_norm_backward(norm, X[:0], None, G[:0])
    assert gx.numel() == 0 and not gw.any() and not gb.any()
    assert ly.tpconv_norm_forward(norm, X[:0]).numel() == 0


def test_norm_gradients_against_differences(ly):
    say("[case] norm gradients against central differences of the definition")
    irreps = "6x0e+5x1o+3x2e"
    x, w, b, g = (v.astype(np.float64) for v in norm_data(irreps, 9, 9))
    norm = ly.Norm(irreps)
    gx, gw, gb = (f64(v) for v in ly.tpconv_norm_backward(norm, cuda(x), cuda(w), cuda(g)))
    loss = lambda x, w, b: float((ol.norm_forward(irreps, x, w, b)[0] * g).sum())
    rng, h = np.random.default_rng(10), 1e-5
    for grad, at in ((gx, 0), (gw, 1), (gb, 2)):
        d = rng.standard_normal(grad.shape)
        lo, hi = ([v - h * d if k == at else v for k, v in enumerate((x, w, b))],
                  [v + h * d if k == at else v for k, v in enumerate((x, w, b))])
        diff = (loss(*hi) - loss(*lo)) / (2 * h)
        # 1e-9 / h of the loss's rounding, h^2 of its third derivative, and the gradient's own tolerance
        assert abs(diff - (grad * d).sum()) <= 1e-4 * np.abs(grad * d).sum()


def test_norm_past_32_bit_offsets(ly):
    import torch

    N, C = 530000, 4096  # 2.17e9 values
    say(f"[case] norm of {N} x {C} bf16 values")
    norm = ly.Norm(f"{C}x0e", 1e-5, ly.TPCONV_BF16, ly.TPCONV_BF16)
    x = torch.zeros((N, C), dtype=torch.bfloat16, device="cuda")
    rows = torch.tensor([0, 1, N // 2, N - 2, N - 1], device="cuda")
    x[rows] = torch.randn((5, C), device="cuda", generator=torch.Generator("cuda").manual_seed(1)).bfloat16()
    y = ly.tpconv_norm_forward(norm, x)
    ref = ol.norm_forward(f"{C}x0e", f64(x[rows]))[0]
    near = 64 * U * 2 * np.abs(ref).max()
    assert np.all(np.abs(f64(y[rows]) - ref) <= near + half_ulp(np.abs(ref) + near))
    assert not y[2:N // 2].any()


# ---- grouped linear layer -------------------------------------------------------------

LINEAR = [("1x0e", "1x0e"), ("3x0e", "5x0e"), ("8x0e+8x1o", "8x0e+8x1o"), ("7x0e+5x1o+3x1o+2x2e", "6x0e+4x1o+3x2e+2x2e"),
          ("33x0e+17x1o", "65x0e+31x1o+2x1e"), ("64x0e+32x1o", "32x0e+64x1o"), ("130x0e+16x2e", "129x0e+24x2e"),
          ("256x0e", "160x0e"), ("40x3o", "36x3o")]


def linear_data(ii, oo, N, G, seed, group=None):
    rng = np.random.default_rng(seed)
    per = ol.linear_blocks(ii, oo)[1]
    group = rng.integers(0, G, N) if group is None else np.asarray(group)
    bf = lambda v: f64(cuda(v, True)).astype(np.float32)
    return (group.astype(np.int32), bf(rng.standard_normal((N, ol.irreps(ii)[1]))), bf(rng.standard_normal((G, per))),
            rng.standard_normal((N, ol.irreps(oo)[1])).astype(np.float32))


def check_linear(ly, ii, oo, G, group, x, W, g, xb=False, wb=False, yb=False, align=True, use_groups=True):
    """x and W are exact in bf16, so every type runs on the same numbers; fp32 runs get fp32 digits on top."""
    import torch

    code = lambda b: ly.TPCONV_BF16 if b else ly.TPCONV_F32
    lin = ly.Linear(ii, oo, G, code(xb), code(wb), code(yb))
    N = len(group)
    if not xb:
        x = x * np.float32(1.2345678)
    if not wb:
        W = W * np.float32(0.7654321)
    X, Wt, Gy = cuda(x, xb), cuda(W, wb), cuda(g)
    if not align:
        X, Wt, Gy = misaligned(X), misaligned(Wt), misaligned(Gy)
    groups = ly.tpconv_linear_groups(lin, torch.from_numpy(group).cuda()) if use_groups else ly.Groups(N)
    if use_groups:
        assert np.array_equal(groups.order.cpu().numpy()[:N], np.argsort(group, kind="stable"))
        assert np.array_equal(np.diff(groups.offsets.cpu().numpy()), np.bincount(group, minlength=G))
    y = ly.tpconv_linear_forward(lin, groups, X, Wt)
    gx, gW = ly.tpconv_linear_backward(lin, groups, X, Wt, Gy)
    gx1, none = ly.tpconv_linear_backward(lin, groups, X, Wt, Gy, want=("x",))
    none2, gW1 = ly.tpconv_linear_backward(lin, groups, X, Wt, Gy, want=("W",))
    torch.cuda.synchronize()
    assert none is None and none2 is None and torch.equal(gx, gx1) and torch.equal(gW, gW1)
    fi, fo = (max([1] + [b[0] for b in ol.irreps(t)[0]]) * len(ol.irreps(t)[0]) for t in (ii, oo))
    near = lambda K: (6 * K / 16 + 16) * U + 2.0 ** -21
    ref, mag = (ol.linear_forward(ii, oo, group, x, W, m) for m in (False, True))
    assert np.all(np.abs(f64(y) - ref) <= near(fi) * mag + (half_ulp(np.abs(ref) + near(fi) * mag) if yb else 0))
    (rx, rW), (mx, mW) = (ol.linear_backward(ii, oo, group, x, W, g, m) for m in (False, True))
    assert np.all(np.abs(f64(gx).reshape(rx.shape) - rx) <= near(fo) * mx)
    assert np.all(np.abs(f64(gW) - rW) <= near(7 * N) * mW)
    return y, gx, gW


@pytest.mark.parametrize("ii,oo", LINEAR)
@pytest.mark.parametrize("xb,wb,yb", [(False, False, False), (True, True, False), (True, True, True),
                                      (True, False, False), (False, True, True)])
def test_linear_matches_definition(ly, ii, oo, xb, wb, yb):
    for N, G in ((1, 1), (1, 5), (37, 4), (150, 3)):
        say(f"[case] linear {ii} -> {oo} N={N} G={G} types {xb}{wb}{yb}")
        check_linear(ly, ii, oo, G, *linear_data(ii, oo, N, G, N + G), xb=xb, wb=wb, yb=yb)


@pytest.mark.parametrize("ii,oo", LINEAR[2:6])
def test_linear_unaligned_and_one_group(ly, ii, oo):
    say(f"[case] linear {ii} -> {oo}, unaligned; then one group without a grouping")
    check_linear(ly, ii, oo, 3, *linear_data(ii, oo, 70, 3, 11), align=False)
    check_linear(ly, ii, oo, 3, *linear_data(ii, oo, 70, 3, 12), xb=True, wb=True, align=False)
    check_linear(ly, ii, oo, 1, *linear_data(ii, oo, 70, 1, 13), use_groups=False)


@pytest.mark.parametrize("N,G,which", [(700, 89, "most empty"), (3, 70, "few"), (1500, 6, "one"), (2000, 2, "uneven"),
                                       (1025, 4096, "more groups than nodes")])
def test_linear_uneven_groups(ly, N, G, which):
    say(f"[case] linear with {N} nodes over {G} groups: {which}")
    rng = np.random.default_rng(14)
    group = {"most empty": lambda: rng.choice([1, 7, 63, 64, 65, 88], N), "few": lambda: np.array([69, 0, 69]),
             "one": lambda: np.full(N, 4), "uneven": lambda: (rng.random(N) < 0.003).astype(int),
             "more groups than nodes": lambda: rng.integers(0, G, N)}[which]()
    ii, oo = ("16x0e+9x1o", "16x0e+8x1o") if G < 1000 else ("4x0e", "8x0e")
    check_linear(ly, ii, oo, G, *linear_data(ii, oo, N, G, 15, group))


def test_linear_wide(ly):
    for xb in (False, True):
        say(f"[case] linear 520x0e -> 392x0e, 300 nodes, bf16 {xb}")
        check_linear(ly, "520x0e", "392x0e", 3, *linear_data("520x0e", "392x0e", 300, 3, 16), xb=xb, wb=xb)
    say("[case] linear 1024x0e -> 512x0e, 2 nodes over 16 groups")
    check_linear(ly, "1024x0e", "512x0e", 16, *linear_data("1024x0e", "512x0e", 2, 16, 17), xb=True, wb=True)


def test_linear_without_pairs_nodes_or_valid_groups(ly):
    import torch
    from equivariant_gnn_tensor_receiver_amd import tpconv as tp

    say("[case] linear without matching irreps, without nodes, with wrong groups")
    lin = ly.Linear("4x0e", "3x1o", 2)
    group = torch.tensor([0, 1, 1], dtype=torch.int32, device="cuda")
    gr = ly.tpconv_linear_groups(lin, group)
    x, W = torch.ones((3, 4), device="cuda"), torch.empty(lin.w_shape, device="cuda")
    assert not ly.tpconv_linear_forward(lin, gr, x, W).any()
    gx, gW = ly.tpconv_linear_backward(lin, gr, x, W, torch.ones((3, 9), device="cuda"))
    assert not gx.any() and gW.numel() == 0
    lin = ly.Linear("4x0e", "4x0e", 2)
    W = torch.ones(lin.w_shape, device="cuda")
    empty = ly.tpconv_linear_groups(lin, group[:0])
    assert empty.offsets.tolist() == [0, 0, 0]
    assert ly.tpconv_linear_forward(lin, empty, x[:0], W).shape == (0, 4)
    gx, gW = ly.tpconv_linear_backward(lin, empty, x[:0], W, x[:0])
    assert gx.numel() == 0 and not gW.any()
    for bad in ([0, 2, 1], [0, -1, 1]):
        ids = torch.tensor(bad, dtype=torch.int32, device="cuda")
        with pytest.raises(tp.TpconvError) as e:
            ly.tpconv_linear_groups(lin, ids)
        assert e.value.status == 3
        left = ly.tpconv_linear_groups(lin, ids, validate=False)  # the node without a group is left out
        y = ly.tpconv_linear_forward(lin, left, x, W, out=torch.full((3, 4), 7.0, device="cuda"))
        assert y.tolist() == [[4.0] * 4, [7.0] * 4, [4.0] * 4]
    with pytest.raises(ValueError):
        ly.tpconv_linear_forward(lin, gr, x.t().contiguous().t(), W)
    with pytest.raises(TypeError):
        ly.tpconv_linear_forward(lin, gr, x.bfloat16(), W)


def test_linear_value_that_is_not_finite_stays_in_its_node_and_group(ly):
    import torch

    say("[case] linear with an infinite and a NaN feature")
    ii = "40x0e+8x1o"
    group, x, W, g = linear_data(ii, ii, 90, 4, 18)
    lin = ly.Linear(ii, ii, 4)
    gr = ly.tpconv_linear_groups(lin, torch.from_numpy(group).cuda())
    y0 = ly.tpconv_linear_forward(lin, gr, cuda(x), cuda(W))
    _, w0 = ly.tpconv_linear_backward(lin, gr, cuda(x), cuda(W), cuda(g))
    x[11, 3], x[12, 45] = np.inf, np.nan
    y1 = ly.tpconv_linear_forward(lin, gr, cuda(x), cuda(W))
    _, w1 = ly.tpconv_linear_backward(lin, gr, cuda(x), cuda(W), cuda(g))
    keep = [v for v in range(90) if v not in (11, 12)]
    assert torch.equal(y0[keep], y1[keep])
    assert not torch.isfinite(y1[11, :40]).any() and torch.equal(y0[11, 40:], y1[11, 40:])
    others = [k for k in range(4) if k not in (group[11], group[12])]
    assert torch.equal(w0[others], w1[others])


def test_linear_gradients_against_differences(ly):
    import torch

    say("[case] linear gradients against central differences of the definition")
    ii, oo = "9x0e+4x1o", "7x0e+6x1o"
    group, x, W, g = linear_data(ii, oo, 30, 3, 19)
    lin = ly.Linear(ii, oo, 3)
    gr = ly.tpconv_linear_groups(lin, torch.from_numpy(group).cuda())
    gx, gW = (f64(v) for v in ly.tpconv_linear_backward(lin, gr, cuda(x), cuda(W), cuda(g)))
    loss = lambda x, W: float((ol.linear_forward(ii, oo, group, x, W) * g).sum())
    rng = np.random.default_rng(20)
    d = rng.standard_normal(x.shape)
    assert abs((loss(x + d, W) - loss(x - d, W)) / 2 - (gx * d).sum()) <= 1e-5 * np.abs(gx * d).sum()
    d = rng.standard_normal(W.shape)
    assert abs((loss(x, W + d) - loss(x, W - d)) / 2 - (gW * d).sum()) <= 1e-5 * np.abs(gW * d).sum()


def test_linear_past_32_bit_offsets(ly):
    import torch

    N, C = 2_200_000, 1024  # 2.25e9 values
    say(f"[case] linear of {N} x {C} bf16 values")
    lin = ly.Linear(f"{C}x0e", "8x0e", 2, ly.TPCONV_BF16, ly.TPCONV_BF16, ly.TPCONV_BF16)
    group = (torch.arange(N, device="cuda") % 2).int()
    gr = ly.tpconv_linear_groups(lin, group)
    x = torch.zeros((N, C), dtype=torch.bfloat16, device="cuda")
    rows = torch.tensor([0, 1, N // 2, N - 2, N - 1], device="cuda")
    gen = torch.Generator("cuda").manual_seed(2)
    x[rows] = torch.randn((5, C), device="cuda", generator=gen).bfloat16()
    W = torch.randn(lin.w_shape, device="cuda", generator=gen).bfloat16()
    y = ly.tpconv_linear_forward(lin, gr, x, W)
    pick = group[rows].cpu().numpy()
    ref, mag = (ol.linear_forward(f"{C}x0e", "8x0e", pick, f64(x[rows]), f64(W), m) for m in (False, True))
    near = ((6 * C / 16 + 16) * U + 2.0 ** -21) * mag
    assert np.all(np.abs(f64(y[rows]) - ref) <= near + half_ulp(np.abs(ref) + near))
    assert not y[2:N // 2].any()


# ---- orthogonalised update --------------------------------------------------------------

QUINTIC = (3.4445, -4.7750, 2.0315)
MUON_TOL = 5 * QUINTIC[0] ** 5 * 2.0 ** -21
SHAPES = [(1, 1), (3, 5), (5, 3), (1, 64), (64, 1), (16, 16), (32, 32), (33, 31), (20, 90), (64, 64), (65, 64),
          (100, 40), (128, 128), (128, 30), (129, 128), (96, 128), (200, 70), (7, 300), (256, 320), (500, 129)]


def frob(a):
    return np.sqrt((np.asarray(a) ** 2).sum((-1, -2)))


def matrices(count, rows, cols, seed, rank=None):
    rng = np.random.default_rng(seed)
    u = rng.standard_normal((count, rows, cols)) * 0.3
    k = max(1, min(rows, cols) // 4)
    return (1e-3 * (u + rng.standard_normal((count, rows, k)) @ rng.standard_normal((count, k, cols)))).astype(np.float32)


@pytest.mark.parametrize("rows,cols", SHAPES)
def test_orthogonalize_matches_definition(ly, rows, cols):
    for count in (1, 3):
        say(f"[case] orthogonalize {count} x {rows} x {cols}")
        u = matrices(count, rows, cols, rows + cols)
        muon = ly.Muon([(rows, cols, count)])
        o = ly.tpconv_muon_orthogonalize(muon, cuda(u))
        assert frob(f64(o) - ol.orthogonalize(u, [QUINTIC] * 5)).max() <= MUON_TOL
        one = ly.tpconv_muon_orthogonalize(ly.Muon([(rows, cols, count)], [QUINTIC]), cuda(u))
        assert frob(f64(one) - ol.orthogonalize(u, [QUINTIC])).max() <= 4 * 2.0 ** -21


@pytest.mark.parametrize("steps", [[(1.5, -0.5, 0.0)] * 3, [(2.0, -1.5, 0.5)] * 16, [(0.0, 0.0, 0.0)], [(1.0, 0.0, 0.0)],
                                   [(30.0, 0.0, 0.0), (0.01, 0.0, 0.0)], [(-1.0, 0.25, -0.125)] * 2])
def test_orthogonalize_other_polynomials(ly, steps):
    for rows, cols in ((24, 40), (150, 130)):
        say(f"[case] orthogonalize {rows} x {cols} with {len(steps)} steps of {steps[0]}")
        u = matrices(2, rows, cols, 21)
        o = ly.tpconv_muon_orthogonalize(ly.Muon([(rows, cols, 2)], steps), cuda(u))
        slope = np.prod([max(1.0, abs(a)) for a, _, _ in steps])
        assert frob(f64(o) - ol.orthogonalize(u, steps)).max() <= len(steps) * slope * 2.0 ** -21 * np.sqrt(24) + 1e-12


def test_orthogonalize_small_large_and_degenerate_matrices(ly):
    import torch

    for rows, cols in ((12, 20), (64, 64), (140, 131)):
        say(f"[case] orthogonalize {rows} x {cols}: zero, tiny, huge, rank one, NaN")
        u = matrices(6, rows, cols, 22)
        u[1] = 0.0
        u[2] *= np.float32(1e-18)   # below eps: X = U / eps
        u[3] *= np.float32(1e17)
        u[4] = np.outer(np.arange(1, rows + 1), np.ones(cols)).astype(np.float32)
        u[5, 0, 0] = np.nan
        muon = ly.Muon([(rows, cols, 6)])
        o = ly.tpconv_muon_orthogonalize(muon, cuda(u))
        assert frob(f64(o[:5]) - ol.orthogonalize(u[:5], [QUINTIC] * 5)).max() <= MUON_TOL
        assert not o[1].any() and torch.isnan(o[5]).all()


@pytest.mark.parametrize("nesterov", [True, False])
def test_muon_step_matches_definition(ly, nesterov):
    import torch

    for rows, cols, count in ((32, 32, 5), (20, 90, 2), (90, 20, 2), (128, 128, 2), (130, 260, 2), (260, 130, 1)):
        say(f"[case] muon step {count} x {rows} x {cols} nesterov={nesterov}")
        rng = np.random.default_rng(23)
        W = rng.standard_normal((count, rows, cols)).astype(np.float32)
        g, m = matrices(count, rows, cols, 24), 0.5 * matrices(count, rows, cols, 25)
        muon = ly.Muon([(rows, cols, count)])
        Wt, M, low = cuda(W), cuda(m), torch.empty((count, rows, cols), dtype=torch.bfloat16, device="cuda")
        args = dict(lr=0.05, beta=0.9, nesterov=nesterov, weight_decay=0.1)
        W1, m1 = ly.tpconv_muon_step(muon, Wt, cuda(g), M, W_bf16=low, **args)
        rW, rm = ol.muon_step(W, g, m, [QUINTIC] * 5, 0.05, 0.9, nesterov, 0.1)
        scale = np.sqrt(max(1.0, cols / rows))
        assert frob(f64(W1) - rW).max() <= 0.05 * scale * MUON_TOL + 4 * U * frob(W).max()
        assert np.abs(f64(m1) - rm).max() <= 4 * U * np.abs(rm).max()
        assert torch.equal(low, W1.bfloat16())
        # in place, and the same result again
        W2, m2 = ly.tpconv_muon_step(muon, Wt, cuda(g), M, W_out=Wt, momentum_out=M, **args)
        assert W2 is Wt and m2 is M and torch.equal(W2, W1) and torch.equal(m2, m1)


def test_muon_blocks_of_several_shapes_with_gaps(ly):
    import torch

    say("[case] muon on banks of several shapes with gaps between them")
    blocks = [(8, 12, 3, 5, 120), (140, 60, 2, 400, 9000), (33, 33, 1, 20000), (5, 4, 0, 30000, 20), (64, 128, 2, 22000, 8192)]
    muon = ly.Muon(blocks)
    rng = np.random.default_rng(26)
    size = 22000 + 2 * 8192 + 11
    u = (rng.standard_normal(size) * 1e-2).astype(np.float32)
    W, g = cuda(rng.standard_normal(size)), cuda(u)
    o = ly.tpconv_muon_orthogonalize(muon, g)
    W1, m1 = ly.tpconv_muon_step(muon, W, g, g, lr=0.1)
    mask = np.zeros(size, bool)
    for rows, cols, count, off, *stride in blocks:
        for i in range(count):
            at = off + i * (stride[0] if stride else rows * cols)
            mask[at:at + rows * cols] = True
            ref = ol.orthogonalize(u[at:at + rows * cols].reshape(rows, cols), [QUINTIC] * 5)
            assert frob(f64(o)[at:at + rows * cols].reshape(rows, cols) - ref) <= MUON_TOL
    rest = torch.from_numpy(~mask).cuda()
    assert not o[rest].any() and torch.equal(W1[rest], W[rest]) and torch.equal(m1[rest], g[rest])
    assert not torch.equal(W1, W)
    # in place: the elements between the blocks stay
    v = g.clone()
    ly.tpconv_muon_orthogonalize(muon, v, out=v)
    assert torch.equal(v[rest], g[rest]) and torch.equal(v[~rest], o[~rest])


# ---- streams, repeats, the layers together ---------------------------------------------------


def test_layers_repeat_bitwise_and_on_another_stream(ly):
    import torch

    say("[case] the layers twice and on a side stream")
    ii = "48x0e+24x1o"
    group, x, W, g = linear_data(ii, ii, 2500, 5, 27)
    norm, lin, muon = ly.Norm(ii), ly.Linear(ii, ii, 5), None
    muon = ly.Muon(ly.weight_blocks(lin) + [(200, 150, 2, 5 * lin.w_per_group)])
    X, Wt, G, gid = cuda(x), cuda(W), cuda(g), torch.from_numpy(group).cuda()
    extra = cuda(matrices(2, 200, 150, 28)).reshape(-1)

    def everything(stream=None):
        gr = ly.tpconv_linear_groups(lin, gid, validate=False, stream=stream)
        y = ly.tpconv_norm_forward(norm, X, stream=stream)
        z = ly.tpconv_linear_forward(lin, gr, y, Wt, stream=stream)
        gy, gW = ly.tpconv_linear_backward(lin, gr, y, Wt, G, stream=stream)
        back = ly.tpconv_norm_backward(norm, X, None, gy, stream=stream)
        if stream is not None:
            stream.synchronize()
        u = torch.cat([gW.reshape(-1), extra])
        return [y, z, gy, gW, *back, ly.tpconv_muon_orthogonalize(muon, u)]

    one, two = everything(), everything()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    three = everything(side)
    torch.cuda.synchronize()
    for a, b, c in zip(one, two, three):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_layers_under_graph_capture(ly):
    """Nothing allocates or synchronises inside the calls, so they can be captured and replayed."""
    import torch

    say("[case] the layers captured into a graph and replayed on new inputs")
    ii = "32x0e+16x1o"
    group, x, W, g = linear_data(ii, ii, 700, 3, 29)
    norm, lin = ly.Norm(ii), ly.Linear(ii, ii, 3)
    muon = ly.Muon(ly.weight_blocks(lin))
    X, Wt, G = cuda(x), cuda(W), cuda(g)
    gr = ly.tpconv_linear_groups(lin, torch.from_numpy(group).cuda())

    def work():
        y = ly.tpconv_norm_forward(norm, X)
        z = ly.tpconv_linear_forward(lin, gr, y, Wt)
        gy, gW = ly.tpconv_linear_backward(lin, gr, y, Wt, G)
        return [z, *ly.tpconv_norm_backward(norm, X, None, gy), ly.tpconv_muon_orthogonalize(muon, gW)]

    work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = work()
    for k in range(3):
        X.copy_(cuda(x * np.float32(1 + k)))
        graph.replay()
        torch.cuda.synchronize()
        got = [v.clone() for v in out]
        for a, b in zip(got, work()):
            assert torch.equal(a, b)
        torch.cuda.synchronize()
