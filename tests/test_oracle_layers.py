"""Pins of the fp64 node layers: differences, equivariance, closed forms, the matrix iteration itself."""
import numpy as np
import pytest

from oracle import layers as ol

QUINTIC = (3.4445, -4.7750, 2.0315)
IRREPS = "5x0e+3x1o+2x0o+4x2e"


def directional(f, x, d, h=1e-5):
    return (f(x + h * d) - f(x - h * d)) / (2 * h)


def test_norm_statistics_and_closed_forms():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((7, ol.irreps(IRREPS)[1])) + 2.0
    y, st = ol.norm_forward(IRREPS, x, eps=1e-12)
    for j, (mul, n, kind, at) in enumerate(ol.irreps(IRREPS)[0]):
        b = y[:, at:at + mul * n]
        assert np.allclose((b * b).mean(1), 1.0)
        assert np.allclose(st[:, j, 0], x[:, at:at + mul * n].mean(1) if kind == "0e" else 0.0)
        if kind == "0e":
            assert np.abs(b.mean(1)).max() < 1e-12
    # a scalar-only string is the usual layer norm
    z, _ = ol.norm_forward("6x0e", x[:, :6], np.arange(6.0), np.ones(6))
    v = x[:, :6]
    assert np.allclose(z, (v - v.mean(1, keepdims=True)) / np.sqrt(v.var(1, keepdims=True) + 1e-5) * np.arange(6) + 1)


def test_norm_is_equivariant():
    rng = np.random.default_rng(1)
    q, _ = np.linalg.qr(rng.standard_normal((3, 3)))  # acts on the rows of a degree-1 block
    x = rng.standard_normal((4, 3, 5))
    w = rng.standard_normal(5)
    a, _ = ol.norm_forward("5x1o", np.einsum("ab,nbc->nac", q, x).reshape(4, -1), w)
    b, _ = ol.norm_forward("5x1o", x.reshape(4, -1), w)
    assert np.allclose(a, np.einsum("ab,nbc->nac", q, b.reshape(4, 3, 5)).reshape(4, -1))


def test_norm_gradients_by_differences():
    rng = np.random.default_rng(2)
    F = ol.irreps(IRREPS)[1]
    x, g = rng.standard_normal((6, F)), rng.standard_normal((6, F))
    w, b = rng.standard_normal(14), rng.standard_normal(5)
    gx, gw, gb = ol.norm_backward(IRREPS, x, w, g)
    loss = lambda x, w, b: float((ol.norm_forward(IRREPS, x, w, b)[0] * g).sum())
    d = rng.standard_normal(x.shape)
    assert np.isclose(directional(lambda v: loss(v, w, b), x, d), (gx * d).sum(), rtol=1e-7)
    d = rng.standard_normal(w.shape)
    assert np.isclose(directional(lambda v: loss(x, v, b), w, d), gw @ d, rtol=1e-7)
    d = rng.standard_normal(b.shape)
    assert np.isclose(directional(lambda v: loss(x, w, v), b, d), gb @ d, rtol=1e-7)


def test_linear_gradients_and_group_selection():
    rng = np.random.default_rng(3)
    ii, oo = "4x0e+3x1o+2x0e", "3x0e+2x1o+2x1e"
    per = ol.linear_blocks(ii, oo)[1]
    assert per == 4 * 3 + 3 * 2 + 2 * 3
    group = np.array([2, 0, 2, 1, 0])
    x, W = rng.standard_normal((5, ol.irreps(ii)[1])), rng.standard_normal((4, per))
    y = ol.linear_forward(ii, oo, group, x, W)
    g = rng.standard_normal(y.shape)
    assert np.abs(y[:, -6:]).max() == 0.0  # 1e has no input
    # one scalar block by hand
    assert np.allclose(y[0, :3], x[0, :4] @ W[2, :12].reshape(4, 3) + x[0, 13:15] @ W[2, 18:].reshape(2, 3))
    gx, gW = ol.linear_backward(ii, oo, group, x, W, g)
    assert np.abs(gW[3]).max() == 0.0
    d = rng.standard_normal(x.shape)
    assert np.isclose((ol.linear_forward(ii, oo, group, d, W) * g).sum(), (gx * d).sum())
    d = rng.standard_normal(W.shape)
    assert np.isclose((ol.linear_forward(ii, oo, group, x, d) * g).sum(), (gW * d).sum())


@pytest.mark.parametrize("rows,cols", [(6, 6), (4, 9), (9, 4), (1, 5)])
def test_orthogonalize_is_the_matrix_iteration(rows, cols):
    rng = np.random.default_rng(4)
    u = rng.standard_normal((rows, cols))
    x = u / np.linalg.norm(u)
    for a, b, c in [QUINTIC] * 5:
        m = x @ x.T
        x = a * x + (b * m + c * m @ m) @ x
    assert np.allclose(x, ol.orthogonalize(u, [QUINTIC] * 5), atol=1e-9)
    # three steps of the cubic 1.5 s - 0.5 s^3 and on converge to the nearest orthogonal matrix
    o = ol.orthogonalize(u, [(1.5, -0.5, 0.0)] * 60)
    e = o @ o.T if rows <= cols else o.T @ o
    assert np.allclose(e, np.eye(min(rows, cols)), atol=1e-8)


def test_muon_step_moves_along_the_orthogonalised_momentum():
    rng = np.random.default_rng(5)
    W, g, m = (rng.standard_normal((2, 3, 12)) for _ in range(3))
    W2, m2 = ol.muon_step(W, g, m, [QUINTIC] * 5, 0.1, 0.9, False, 0.5)
    assert np.allclose(m2, 0.9 * m + 0.1 * g)
    assert np.allclose((0.95 * W - W2) / 0.1, 2.0 * ol.orthogonalize(m2, [QUINTIC] * 5))
