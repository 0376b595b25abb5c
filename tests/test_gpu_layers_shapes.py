"""GPU parity of the node layers in every tile shape and row width that a call of real size takes.

Each case names the kernels that it is meant to reach and fails if the library took others (names of the traced
launches), so that a changed rule of choice cannot leave a shape without a comparison.  Tolerances are those of
test_gpu_layers.py; a weight gradient's sum is split into slots of at most 1024 rows at these sizes, whose sums are
added in order: 6 * 1024 / 16 roundings within a slot and one per slot of 128 rows or more.
"""
import warnings

import numpy as np
import pytest

from gpu_cases import say
from oracle import layers as ol
from test_gpu_layers import (MUON_TOL, QUINTIC, U, check_norm, cuda, f64, frob, half_ulp, ly, matrices,  # noqa: F401
                             misaligned, norm_data)

pytestmark = pytest.mark.gpu


def launched(fn):
    """fn() and the names of the kernels that it launched."""
    import torch
    from torch.profiler import ProfilerActivity, profile

    torch.cuda.synchronize()
    with warnings.catch_warnings():
        warnings.simplefilter("ignore")
        with profile(activities=[ProfilerActivity.CUDA]) as p:
            out = fn()
            torch.cuda.synchronize()
        names = {e.name for e in p.events()}
    return out, {n.replace("tpconv::", "").replace("(anonymous namespace)::", "") for n in names if "tpconv::" in n}


def reached(names, *parts):
    """Whether one kernel's name holds all the parts, in order."""
    for n in names:
        at = 0
        for p in parts:
            at = n.find(p, at)
            if at < 0:
                break
            at += len(p)
        else:
            return True
    return False


# ---- grouped linear layer ---------------------------------------------------------------


def grouped(ii, oo, group, x, W, g, magnitude=False):
    """y, gx, gW group by group in 64 bits (or the sums of the terms' magnitudes)."""
    blocks, per = ol.linear_blocks(ii, oo)
    x, W, g = (np.asarray(v, dtype=np.float64) for v in (x, W, g))
    if magnitude:
        x, W, g = np.abs(x), np.abs(W), np.abs(g)
    y, gx, gW = np.zeros_like(g), np.zeros_like(x), np.zeros_like(W)
    for e in np.unique(group):
        v = np.flatnonzero(group == e)
        xe, ge, ye, gxe = x[v], g[v], y[v], gx[v]
        for (mi, n, _, xi), (mo, _, _, yo), at in blocks:
            w = W[e, at:at + mi * mo].reshape(mi, mo)
            a, b = xe[:, xi:xi + n * mi].reshape(-1, mi), ge[:, yo:yo + n * mo].reshape(-1, mo)
            ye[:, yo:yo + n * mo] += (a @ w).reshape(len(v), -1)
            gxe[:, xi:xi + n * mi] += (b @ w.T).reshape(len(v), -1)
            gW[e, at:at + mi * mo] += (a.T @ b).ravel()
        y[v], gx[v] = ye, gxe
    return y, gx, gW


def test_grouped_definition_is_the_oracles():
    ii, oo = "5x0e+3x1o+2x1o", "4x0e+6x1o"
    rng = np.random.default_rng(50)
    group, W = rng.integers(0, 3, 20), rng.standard_normal((3, ol.linear_blocks(ii, oo)[1]))
    x, g = rng.standard_normal((20, ol.irreps(ii)[1])), rng.standard_normal((20, ol.irreps(oo)[1]))
    for m in (False, True):
        want = (ol.linear_forward(ii, oo, group, x, W, m), *ol.linear_backward(ii, oo, group, x, W, g, m))
        assert all(np.allclose(a, b, rtol=1e-13, atol=1e-13) for a, b in zip(grouped(ii, oo, group, x, W, g, m), want))


ROWS = {128: "Shape<128, 128,", 64: "Shape<128, 64,", 32: "Shape<128, 32,", 0: "Shape<32, 32,"}
GW = {128: "Shape<128, 128,", 64: "Shape<64, 64,", 32: "Shape<32, 32,"}
# irreps, nodes, groups (0: one, without a grouping), column widths of the forward, of the input gradient and of the
# weight gradient's tiles (0: the shape for few rows)
LINEAR = [
    ("121x3o", "121x3o", 5000, 7, 128, 128, 128),
    ("29x3o", "121x3o", 5000, 7, 128, 32, 64),
    ("121x3o", "29x3o", 5000, 7, 32, 128, 64),
    ("61x3o", "61x3o", 5000, 7, 64, 64, 64),
    ("29x3o", "29x3o", 5000, 7, 32, 32, 32),
    ("61x3o+29x0e", "29x0e", 5000, 7, 0, 64, 32),
    ("121x3o+29x0e", "29x0e+5x2e", 5000, 7, 32, 128, 32),
    ("121x0e", "121x0e", 9001, 11, 32, 32, 128),
    ("121x1o", "121x1o", 6000, 100, 64, 64, 128),
    ("128x3o", "128x3o", 5000, 3, 128, 128, 128),
    ("200x3o", "250x3o", 6000, 5, 128, 128, 128),      # slots of 512 rows: the table of row addresses is refilled
    ("512x0e", "256x0e", 20011, 4, 128, 128, 128),     # the same, tiles dealt out over the XCDs
    ("65x0e+33x1o+20x1o+17x2e", "48x0e+40x1o+24x2e+7x2e", 5003, 89, 32, 32, 32),
    ("100x2e", "72x2e+8x2e", 9000, 0, 32, 128, 128),
]


@pytest.mark.parametrize("ii,oo,N,G,fw,bw,gw", LINEAR)
@pytest.mark.parametrize("xb,wb,yb", [(False, False, False), (True, True, False), (True, True, True),
                                      (True, False, False), (False, True, True)])
def test_linear_wide_shapes(ly, ii, oo, N, G, fw, bw, gw, xb, wb, yb):
    import torch

    say(f"[case] linear {ii} -> {oo} N={N} G={G} types {xb}{wb}{yb}")
    rng = np.random.default_rng(51)
    n_groups, per = max(G, 1), ol.linear_blocks(ii, oo)[1]
    share = 1.0 / (np.arange(n_groups) + 2.0) ** 2 * (np.arange(n_groups) % 5 != 3)  # uneven, some without nodes
    group = rng.choice(n_groups, N, p=share / share.sum()).astype(np.int32)
    code = lambda b: ly.TPCONV_BF16 if b else ly.TPCONV_F32
    lin = ly.Linear(ii, oo, n_groups, code(xb), code(wb), code(yb))
    X, Wt, Gy = (cuda(rng.standard_normal(s), b) for s, b in (((N, lin.feat_in), xb), ((n_groups, per), wb),
                                                              ((N, lin.feat_out), False)))
    if N % 2:
        X, Wt, Gy = misaligned(X), misaligned(Wt), misaligned(Gy)
    x, W, g = f64(X), f64(Wt), f64(Gy)
    groups = ly.tpconv_linear_groups(lin, torch.from_numpy(group).cuda()) if G else ly.Groups(N)
    y, forward = launched(lambda: ly.tpconv_linear_forward(lin, groups, X, Wt))
    (gx, gW), backward = launched(lambda: ly.tpconv_linear_backward(lin, groups, X, Wt, Gy))
    assert reached(forward, "lin_rows_kernel<" + ROWS[fw]), forward
    assert reached(backward, "lin_backward_kernel<" + ROWS[bw], GW[gw]), backward
    gx1, _ = ly.tpconv_linear_backward(lin, groups, X, Wt, Gy, want=("x",))
    _, gW1 = ly.tpconv_linear_backward(lin, groups, X, Wt, Gy, want=("W",))
    assert torch.equal(gx, gx1) and torch.equal(gW, gW1)
    near = lambda K: (6 * K / 16 + 16) * U + 2.0 ** -21
    longest = lambda text: sum(b[0] for b in ol.irreps(text)[0])
    (ry, rx, rW), (my, mx, mW) = (grouped(ii, oo, group, x, W, g, m) for m in (False, True))
    assert np.all(np.abs(f64(y) - ry) <= near(longest(ii)) * my + (half_ulp(np.abs(ry) + near(longest(ii)) * my) if yb else 0))
    assert np.all(np.abs(f64(gx) - rx) <= near(longest(oo)) * mx)
    assert np.all(np.abs(f64(gW) - rW) <= (near(1024) + 7 * N / 128 * U) * mW)


# ---- orthogonalised update ----------------------------------------------------------------

# count, rows, cols, tile widths of the r x r products and of B X
MUON = [(48, 256, 256, 128, 128), (48, 300, 200, 128, 128), (64, 129, 131, 128, 128), (14, 250, 1000, 64, 128),
        (44, 250, 250, 128, 64), (6, 700, 520, 64, 64), (7, 520, 700, 64, 128)]


@pytest.mark.parametrize("count,rows,cols,square,apply", MUON)
def test_muon_wide_tiles(ly, count, rows, cols, square, apply):
    import torch

    say(f"[case] muon {count} x {rows} x {cols}")
    muon, u = ly.Muon([(rows, cols, count)]), matrices(count, rows, cols, 52)
    o, names = launched(lambda: ly.tpconv_muon_orthogonalize(muon, cuda(u)))
    for phase, width in ((0, square), (1, square), (2, apply), (3, apply)):
        assert reached(names, f"muon_gemm_kernel<{phase}, {width}>"), names
    assert frob(f64(o) - ol.orthogonalize(u, [QUINTIC] * 5)).max() <= MUON_TOL
    one = ly.tpconv_muon_orthogonalize(ly.Muon([(rows, cols, count)], [QUINTIC]), cuda(u))
    assert frob(f64(one) - ol.orthogonalize(u, [QUINTIC])).max() <= 4 * 2.0 ** -21
    rng = np.random.default_rng(53)
    W, m = rng.standard_normal((count, rows, cols)).astype(np.float32), 0.5 * matrices(count, rows, cols, 54)
    low = torch.empty((count, rows, cols), dtype=torch.bfloat16, device="cuda")
    W1, m1 = ly.tpconv_muon_step(muon, cuda(W), cuda(u), cuda(m), lr=0.05, beta=0.9, nesterov=True, weight_decay=0.1,
                                 W_bf16=low)
    rW, rm = ol.muon_step(W, u, m, [QUINTIC] * 5, 0.05, 0.9, True, 0.1)
    scale = np.sqrt(max(1.0, cols / rows))
    assert frob(f64(W1) - rW).max() <= 0.05 * scale * MUON_TOL + 4 * U * frob(W).max()
    assert np.abs(f64(m1) - rm).max() <= 4 * U * np.abs(rm).max()
    assert torch.equal(low, W1.bfloat16())


# ---- layer norm ---------------------------------------------------------------------------

# irreps, nodes, the forward's kernel
NORM = [("259x0e", 700, "wide_kernel<1,"), ("700x0o", 700, "wide_kernel<1,"), ("1500x0e", 1100, "wide_kernel<2,"),
        ("3001x0e", 1100, "wide_kernel<4,"), ("4099x0e", 40, "wide_kernel<8,"), ("5000x0e", 1100, "wide_kernel<8,"),
        ("8191x0e", 600, "wide_kernel<8,"), ("8192x0e", 7, "wide_kernel<8,"), ("6001x0o", 30, "wide_kernel<8,"),
        ("4097x0o+5x1o", 30, "wide_kernel<8,"), ("300x1o+8193x0e", 600, "norm_forward_kernel<"),
        ("7x0e+5x1o", 300000, "narrow_kernel<"), ("32x0e+32x1o+32x2e", 50001, "narrow_kernel<"),
        ("130x0o+3x3o", 9000, "narrow_kernel<")]


@pytest.mark.parametrize("irreps,N,kernel", NORM)
@pytest.mark.parametrize("bf16", [False, True])
def test_norm_row_widths_and_many_trips(ly, irreps, N, kernel, bf16):
    """Every width of the wide kernels, with and without a remainder, and more nodes than the blocks of a launch take
    at a time."""
    say(f"[case] norm {irreps} N={N} bf16={bf16}")
    data = norm_data(irreps, N, 55)
    x, w, b, g = data
    norm = ly.Norm(irreps, 1e-5, *([ly.TPCONV_BF16] * 2 if bf16 else []))
    X, Wt, B, G = cuda(x, bf16), cuda(w), cuda(b), cuda(g)
    _, names = launched(lambda: ly.tpconv_norm_forward(norm, X, Wt, B))
    assert reached(names, "norm_forward", kernel.split("norm_forward")[-1]), names
    _, names = launched(lambda: ly.tpconv_norm_backward(norm, X, Wt, G))
    back = kernel.split("norm_forward")[-1]
    assert reached(names, "norm_backward", back) and reached(names, "norm_reduce_kernel"), names
    check_norm(ly, irreps, *data, xb=bf16, yb=bf16, align=N % 2 == 0)


def test_norm_forward_more_nodes_than_blocks(ly):
    import torch

    N, irreps = 270001, "130x0e"  # four nodes per block and trip, 65536 blocks
    say(f"[case] norm {irreps} N={N}")
    norm = ly.Norm(irreps)
    gen = torch.Generator("cuda").manual_seed(56)
    x = torch.randn((N, 130), device="cuda", generator=gen)
    stats = torch.full(norm.stats_shape(N), float("nan"), device="cuda")
    y = ly.tpconv_norm_forward(norm, x, stats=stats)
    rows = torch.cat([torch.tensor([0, 262143, 262144, N - 1], device="cuda"),
                      torch.randint(0, N, (3000,), device="cuda", generator=gen)])
    ref, st = ol.norm_forward(irreps, f64(x[rows]))
    assert np.abs(f64(y[rows]) - ref).max() <= 64 * U * 2 * np.abs(ref).max()
    assert np.abs(f64(stats[rows]) - st).max() <= 64 * U * 2 * np.abs(st).max()
    assert torch.isfinite(y).all() and torch.isfinite(stats).all()
