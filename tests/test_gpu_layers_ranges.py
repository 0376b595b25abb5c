"""The node layers at the ends of the range of fp32 and on empty tensors, against their fp64 definitions.

The orthogonalisation's tolerances are those of test_gpu_layers.py: a matrix's scale takes no part in them.
"""
import numpy as np
import pytest

from gpu_cases import say
from oracle import layers as ol
from test_gpu_layers import MUON_TOL, QUINTIC, U, cuda, f64, frob, ly, matrices  # noqa: F401  (ly: the fixture)

pytestmark = pytest.mark.gpu

# one block of threads per matrix (both tile sizes, transposed), and the tiled path (T = 64, transposed)
MUON_SHAPES = [(32, 32), (12, 40), (100, 90), (140, 131), (131, 300), (300, 131)]


def scaled(count, rows, cols, seed, largest):
    """Matrices whose largest entry is `largest` in magnitude."""
    u = matrices(count, rows, cols, seed).astype(np.float64)
    return (u / np.abs(u).max((1, 2), keepdims=True) * largest).astype(np.float32)


@pytest.mark.parametrize("rows,cols", MUON_SHAPES)
def test_orthogonalize_any_finite_matrix(ly, rows, cols):
    """Entries whose squares leave fp32 on either side: the singular values are those of the scaled matrix."""
    for largest in (9e17, 1e19, 1e30, 3.4e38):
        say(f"[case] orthogonalize {rows} x {cols} with entries of {largest:g}")
        u = scaled(2, rows, cols, 31, largest)
        o = ly.tpconv_muon_orthogonalize(ly.Muon([(rows, cols, 2)]), cuda(u))
        assert frob(f64(o) - ol.orthogonalize(u, [QUINTIC] * 5)).max() <= MUON_TOL
    for largest, eps in ((1e-20, 1e-30), (1e-30, 1e-40), (1e-38, 1e-45), (1e-30, 1e-7), (1e30, 1e-45)):
        say(f"[case] orthogonalize {rows} x {cols} with entries of {largest:g} and eps {eps:g}")
        u = scaled(2, rows, cols, 32, largest)
        u[1] = 0.0
        o = ly.tpconv_muon_orthogonalize(ly.Muon([(rows, cols, 2)], eps=eps), cuda(u))
        least = float(np.float32(eps))
        assert frob(f64(o) - ol.orthogonalize(u, [QUINTIC] * 5, least)).max() <= MUON_TOL
        assert not o[1].any()


def test_orthogonalize_parts_of_very_different_size(ly):
    """Rows of zeros, tiny and huge entries in one matrix: the chunks of its norm have different scales."""
    for eps in (1e-7, 1e-45):
        say(f"[case] orthogonalize 400 x 150 with rows of different scales, eps {eps:g}")
        u = matrices(2, 400, 150, 33)
        u[:, :30] = 0.0
        u[:, 30:60] *= np.float32(1e-30)
        u[0, 390:] *= np.float32(1e33)
        u[1, 390:] *= np.float32(1e22)
        o = ly.tpconv_muon_orthogonalize(ly.Muon([(400, 150, 2)], eps=eps), cuda(u))
        assert frob(f64(o) - ol.orthogonalize(u, [QUINTIC] * 5, eps)).max() <= MUON_TOL


@pytest.mark.parametrize("rows,cols", [(32, 32), (140, 131)])
@pytest.mark.parametrize("nesterov", [True, False])
def test_muon_step_with_huge_gradients(ly, rows, cols, nesterov):
    say(f"[case] muon step {rows} x {cols} with gradients of 1e30")
    W = np.random.default_rng(34).standard_normal((2, rows, cols)).astype(np.float32)
    g, m = scaled(2, rows, cols, 35, 1e30), scaled(2, rows, cols, 36, 3e29)
    W1, m1 = ly.tpconv_muon_step(ly.Muon([(rows, cols, 2)]), cuda(W), cuda(g), cuda(m), lr=0.05, beta=0.9,
                                 nesterov=nesterov, weight_decay=0.1)
    rW, rm = ol.muon_step(W, g, m, [QUINTIC] * 5, 0.05, 0.9, nesterov, 0.1)
    scale = np.sqrt(max(1.0, cols / rows))
    assert frob(f64(W1) - rW).max() <= 0.05 * scale * MUON_TOL + 4 * U * frob(W).max()
    assert np.abs(f64(m1) - rm).max() <= 4 * U * np.abs(rm).max()
    assert not np.array_equal(f64(W1), np.float64(np.float32(1 - 0.005)) * W)  # more than the decay


def test_orthogonalize_infinite_entry_is_not_hidden(ly):
    import torch

    for rows, cols in ((12, 40), (140, 131)):
        say(f"[case] orthogonalize {rows} x {cols} with an infinite entry")
        u = matrices(2, rows, cols, 37)
        u[1, 3, 4] = np.inf
        o = ly.tpconv_muon_orthogonalize(ly.Muon([(rows, cols, 2)]), cuda(u))
        assert torch.isfinite(o[0]).all() and torch.isnan(o[1]).all()


def test_gradients_of_empty_tensors(ly):
    """Gradients asked for one at a time where there is nothing to compute: no nodes, no 0e block, no pair of irreps."""
    import torch

    say("[case] empty gradients, one at a time")
    dev = torch.device("cuda")
    norm, odd = ly.Norm("8x0e+8x1o"), ly.Norm("4x1o")
    x, three = torch.zeros(0, 32, device=dev), torch.ones(3, 12, device=dev)
    for name in ("x", "weight", "bias"):
        got = dict(zip(("x", "weight", "bias"), ly.tpconv_norm_backward(norm, x, None, x, want=(name,))))
        assert [k for k, v in got.items() if v is not None] == [name] and not got[name].any()
    assert ly.tpconv_norm_backward(odd, three, None, three, want=("bias",))[2].numel() == 0
    lin, none = ly.Linear("4x0e", "3x0e", 2), ly.Linear("4x0e", "3x1o", 2)
    nobody = ly.tpconv_linear_groups(lin, torch.zeros(0, dtype=torch.int32, device=dev))
    W = torch.ones(lin.w_shape, device=dev)
    gx, gW = ly.tpconv_linear_backward(lin, nobody, x.view(0, 4), W, x.view(0, 3), want=("x",))
    assert gx.shape == (0, 4) and gW is None
    gx, gW = ly.tpconv_linear_backward(lin, nobody, x.view(0, 4), W, x.view(0, 3), want=("W",))
    assert gx is None and not gW.any()
    groups = ly.tpconv_linear_groups(none, torch.zeros(3, dtype=torch.int32, device=dev))
    gx, gW = ly.tpconv_linear_backward(none, groups, torch.ones(3, 4, device=dev), torch.zeros(none.w_shape, device=dev),
                                       torch.ones(3, 9, device=dev), want=("W",))
    assert gx is None and gW.shape == (2, 0)
    u = torch.zeros(0, 4, 4, device=dev)
    assert ly.tpconv_muon_orthogonalize(ly.Muon([(4, 4, 0)]), u).shape == (0, 4, 4)


def test_results_on_another_stream_have_memory_of_their_own(ly):
    """A block that the current stream has just given back is not handed to a call on another stream."""
    import torch

    say("[case] results of calls on a side stream")
    side = torch.cuda.Stream()
    norm, lin = ly.Norm("40x0e+8x1o"), ly.Linear("40x0e+8x1o", "40x0e+8x1o", 2)
    x = torch.randn(50000, 64, device="cuda")
    W = torch.randn(lin.w_shape, device="cuda")
    groups = ly.tpconv_linear_groups(lin, torch.zeros(50000, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    want = ly.tpconv_norm_forward(norm, x), ly.tpconv_linear_forward(lin, groups, x, W)
    torch.cuda.synchronize()
    for call, ref in ((lambda: ly.tpconv_norm_forward(norm, x, stream=side), want[0]),
                      (lambda: ly.tpconv_linear_forward(lin, groups, x, W, stream=side), want[1])):
        given_back = torch.empty_like(x)
        address = given_back.data_ptr()
        del given_back
        y = call()
        assert y.data_ptr() != address and torch.empty_like(x).data_ptr() == address
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(y, ref)


def test_linear_products_within_their_bound(ly):
    """Single products of fp32 operands whose three pieces are all as large as they can be (the products left out come
    to 1.96 * 2^-22 of the term), as small as they can be, and at the end of the range: 2^-21, and six roundings."""
    import torch

    say("[case] linear: single products of the worst bit patterns")
    bits = [0x3F80FFFF, 0xBF80FFFF, 0x3FFFFFFF, 0x3F800000, 0x3F810001, 0x3F80FF01, 0x7F7FFFFF, 0x5F80FFFF, 0x2080FFFF]
    v = np.array(bits, dtype=np.uint32).view(np.float32)
    w = np.array([0x3F80FFFF, 0xBFFFFFFF, 0x3F808080, 0x3F000001], dtype=np.uint32).view(np.float32)
    lin = ly.Linear("1x0e", "1x0e")
    x = torch.from_numpy(v.copy()).cuda().view(-1, 1)
    for one in w:
        W = torch.full(lin.w_shape, float(one), device="cuda")
        y = ly.tpconv_linear_forward(lin, ly.Groups(len(v)), x, W)
        gx, _ = ly.tpconv_linear_backward(lin, ly.Groups(len(v)), x, W, x, want=("x",))
        ref = v.astype(np.float64) * np.float64(one)
        fits = np.abs(ref) < 3.4e38
        for got in (y, gx):
            assert np.all(np.abs(f64(got)[fits, 0] - ref[fits]) <= (2.0 ** -21 + 6 * U) * np.abs(ref[fits]))
    # bf16 x fp32: every product of the pieces is kept
    half = ly.Linear("1x0e", "1x0e", 1, ly.TPCONV_BF16)
    xb = x.bfloat16()
    keep = torch.isfinite(xb[:, 0]).cpu().numpy()
    for one in w:
        y = ly.tpconv_linear_forward(half, ly.Groups(len(v)), xb, torch.full(half.w_shape, float(one), device="cuda"))
        ref = f64(xb)[:, 0] * np.float64(one)
        keep = keep & (np.abs(ref) < 3.4e38)
        assert np.all(np.abs(f64(y)[keep, 0] - ref[keep]) <= 3 * U * np.abs(ref[keep]))


@pytest.mark.parametrize("sizes", [[128, 129, 127, 0, 256, 257, 0, 1] + [0] * 40, [0] * 300 + [130], [129] * 9, [5000, 0, 1],
                                   [64] * 100 + [500] + [3] * 50, [128] * 4, [1] * 70])
def test_weight_gradient_partial_sums_stay_in_their_workspace(ly, sizes):
    """Groups of one slot and of several, with many groups and few: a workspace of exactly the size asked for."""
    import torch
    from test_gpu_layers_shapes import grouped

    ii, oo, G, N = "9x0e+5x1o", "7x0e+6x1o", len(sizes), sum(sizes)
    say(f"[case] linear weight gradient of {N} nodes in {G} groups, the largest of {max(sizes)}")
    lin, rng = ly.Linear(ii, oo, G), np.random.default_rng(38)
    group = rng.permutation(np.repeat(np.arange(G), sizes)).astype(np.int32)
    x, W, g = (rng.standard_normal(s).astype(np.float32) for s in ((N, lin.feat_in), lin.w_shape, (N, lin.feat_out)))
    groups = ly.tpconv_linear_groups(lin, torch.from_numpy(group).cuda())
    size = lin.workspace_size(N)
    memory = torch.full((size + 4096,), 77, dtype=torch.uint8, device="cuda")
    gx, gW = ly.tpconv_linear_backward(lin, groups, cuda(x), cuda(W), cuda(g), workspace=memory[:size])
    assert (memory[size:] == 77).all()
    (_, rx, rW), (_, mx, mW) = (grouped(ii, oo, group, x, W, g, m) for m in (False, True))
    near = lambda K: (6 * K / 16 + 16) * U + 2.0 ** -21
    assert np.all(np.abs(f64(gx) - rx) <= near(13) * mx)
    assert np.all(np.abs(f64(gW) - rW) <= near(3 * max(sizes)) * mW)
