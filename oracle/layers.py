"""fp64 definitions of the node layers: layer norm over irreps, the grouped linear layer, the orthogonalised update.

Plain numpy, written from the formulas: the norm's gradient through its Jacobian's projections, the linear layer node by
node, the orthogonalisation through the singular values (an odd polynomial of a matrix acts on them alone).
"""
from __future__ import annotations

import re

import numpy as np


def irreps(text):
    """[(mul, 2l+1, kind such as "0e", feature offset)] and the features per node."""
    out, at = [], 0
    for mul, l, p in re.findall(r"(\d+)x(\d+)([eo])", text.replace(" ", "")):
        n = 2 * int(l) + 1
        out.append((int(mul), n, l + p, at))
        at += int(mul) * n
    return out, at


def norm_forward(text, x, weight=None, bias=None, eps=1e-5):
    """y and the statistics [N][irreps][2]."""
    blocks, F = irreps(text)
    x = np.asarray(x, dtype=np.float64).reshape(-1, F)
    y, stats, wo, bo = np.empty_like(x), np.zeros((x.shape[0], len(blocks), 2)), 0, 0
    for j, (mul, n, kind, at) in enumerate(blocks):
        v = x[:, at:at + mul * n].reshape(-1, n, mul)
        mu = v.mean(axis=(1, 2)) if kind == "0e" else np.zeros(x.shape[0])
        d = v - mu[:, None, None]
        r = 1.0 / np.sqrt((d * d).mean(axis=(1, 2)) + eps)
        z = d * r[:, None, None]
        if weight is not None:
            z = z * weight[wo:wo + mul]
        if kind == "0e" and bias is not None:
            z = z + bias[bo:bo + mul]
        wo += mul
        bo += mul if kind == "0e" else 0
        y[:, at:at + mul * n] = z.reshape(-1, n * mul)
        stats[:, j, 0], stats[:, j, 1] = mu, r
    return y, stats


def norm_backward(text, x, weight, g, eps=1e-5):
    """grad_x, grad_weight, grad_bias of <g, y>.  With u the (centred) block and s^2 = |u|^2 + n eps, y / w is
    sqrt(n) u / s, whose Jacobian is sqrt(n) / s (1 - u u^T / s^2) on the centred space."""
    blocks, F = irreps(text)
    x = np.asarray(x, dtype=np.float64).reshape(-1, F)
    g = np.asarray(g, dtype=np.float64).reshape(-1, F)
    gx, gw, gb, wo = np.empty_like(x), [], [], 0
    for mul, n, kind, at in blocks:
        size = mul * n
        u, h = x[:, at:at + size], g[:, at:at + size]
        w = np.ones(size) if weight is None else np.tile(np.asarray(weight, dtype=np.float64)[wo:wo + mul], n)
        wo += mul
        if kind == "0e":
            u = u - u.mean(1, keepdims=True)
        s = np.sqrt((u * u).sum(1, keepdims=True) + size * eps)
        gw.append((h * u / s * np.sqrt(size)).sum(0).reshape(n, mul).sum(0))
        if kind == "0e":
            gb.append(h.sum(0))
        t = h * w
        t = np.sqrt(size) / s * (t - u * (t * u).sum(1, keepdims=True) / s ** 2)
        gx[:, at:at + size] = t - t.mean(1, keepdims=True) if kind == "0e" else t
    return gx, np.concatenate(gw), np.concatenate(gb) if gb else np.zeros(0)


def linear_blocks(irreps_in, irreps_out):
    """[(input block, output block, offset)] of equal degree and parity, and the weights per group."""
    out, at = [], 0
    for i in irreps(irreps_in)[0]:
        for o in irreps(irreps_out)[0]:
            if i[2] == o[2]:
                out.append((i, o, at))
                at += i[0] * o[0]
    return out, at


def linear_forward(irreps_in, irreps_out, group, x, W, magnitude=False):
    """y [N][F_out]; magnitude: the sum of the terms' magnitudes instead (what rounding errors scale with)."""
    blocks, per = linear_blocks(irreps_in, irreps_out)
    Fi, Fo = irreps(irreps_in)[1], irreps(irreps_out)[1]
    x, W = np.asarray(x, dtype=np.float64).reshape(-1, Fi), np.asarray(W, dtype=np.float64).reshape(-1, per)
    if magnitude:
        x, W = np.abs(x), np.abs(W)
    y = np.zeros((x.shape[0], Fo))
    for v in range(x.shape[0]):
        for (mi, n, _, xi), (mo, _, _, yo), at in blocks:
            w = W[group[v], at:at + mi * mo].reshape(mi, mo)
            y[v, yo:yo + n * mo] += (x[v, xi:xi + n * mi].reshape(n, mi) @ w).ravel()
    return y


def linear_backward(irreps_in, irreps_out, group, x, W, g, magnitude=False):
    """grad_x, grad_W of <g, y> (or the sums of the terms' magnitudes)."""
    blocks, per = linear_blocks(irreps_in, irreps_out)
    Fi, Fo = irreps(irreps_in)[1], irreps(irreps_out)[1]
    x, W = np.asarray(x, dtype=np.float64).reshape(-1, Fi), np.asarray(W, dtype=np.float64).reshape(-1, per)
    g = np.asarray(g, dtype=np.float64).reshape(-1, Fo)
    if magnitude:
        x, W, g = np.abs(x), np.abs(W), np.abs(g)
    gx, gW = np.zeros_like(x), np.zeros_like(W)
    for v in range(x.shape[0]):
        for (mi, n, _, xi), (mo, _, _, yo), at in blocks:
            w = W[group[v], at:at + mi * mo].reshape(mi, mo)
            gv, xv = g[v, yo:yo + n * mo].reshape(n, mo), x[v, xi:xi + n * mi].reshape(n, mi)
            gx[v, xi:xi + n * mi] += (gv @ w.T).ravel()
            gW[group[v], at:at + mi * mo] += (xv.T @ gv).ravel()
    return gx, gW


def orthogonalize(u, steps, eps=1e-7):
    """The matrices u [..][rows][cols] with the singular values mapped by the steps' polynomials."""
    left, s, right = np.linalg.svd(np.asarray(u, dtype=np.float64), full_matrices=False)
    s = s / np.maximum(np.sqrt((s * s).sum(-1, keepdims=True)), eps)
    for a, b, c in steps:
        s = s * (a + s ** 2 * (b + c * s ** 2))
    return (left * s[..., None, :]) @ right


def muon_step(W, grad, momentum, steps, lr, beta, nesterov, weight_decay, eps=1e-7):
    """New weights and momentum of matrices [..][rows][cols] (rows: inputs, cols: outputs)."""
    W, grad, m = (np.asarray(v, dtype=np.float64) for v in (W, grad, momentum))
    m = beta * m + (1 - beta) * grad
    u = (1 - beta) * grad + beta * m if nesterov else m
    scale = np.sqrt(max(1.0, W.shape[-1] / W.shape[-2]))
    return (1 - lr * weight_decay) * W - lr * scale * orthogonalize(u, steps, eps), m
