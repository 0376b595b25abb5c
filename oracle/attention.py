"""fp64 definitions of the attention block's operators on numpy arrays: attention among the nodes of each graph (its
gradients by the chain rule on the full score matrices), the embedding of node types, and dropout from Philox4x32-10.

Node tensors are [N][F], per node the blocks [2l+1][mul] of the irreps string in order.  Test infrastructure only; shares
no code with the library.
"""
from __future__ import annotations

import numpy as np

from .layers import irreps


def head_columns(text, heads):
    """For every head the columns of a node tensor that belong to it."""
    got = []
    for h in range(heads):
        c = []
        for mul, n, _, at in irreps(text)[0]:
            per = mul // heads
            for r in range(n):
                c += range(at + r * mul + h * per, at + r * mul + (h + 1) * per)
        got.append(np.array(c, dtype=np.int64))
    return got


def scores(q, k, scale, cap, slope, rq, rk):
    """(scores, tanh of capped ones or None, distances or None) of one graph and head."""
    s = scale * (q @ k.T)
    th = None
    if cap > 0:
        th = np.tanh(s / cap)
        s = cap * th
    d = None
    if slope is not None:
        d = np.sqrt(((rq[:, None] - rk[None]) ** 2).sum(-1))
        s = s - slope * d
    return s, th, d


def attention(irreps_qk, irreps_v, heads, q, k, v, offsets, key_offsets=None, scale=1.0, cap=0.0, slope=None, pos=None,
              key_pos=None, grad_out=None):
    """out, or with grad_out a dict of out, lse (base 2), grad_q, grad_k, grad_v, grad_slope, grad_pos, grad_key_pos (self
    form: grad_pos holds both ends), and abs_*: bounds of the sums of the magnitudes of the terms of out and the gradients."""
    cross = key_offsets is not None
    ko = key_offsets if cross else offsets
    kp = key_pos if cross else pos
    cq, cv = head_columns(irreps_qk, heads), head_columns(irreps_v, heads)
    z = np.zeros
    o = dict(out=z((q.shape[0], v.shape[1])), lse=np.full((heads, q.shape[0]), -np.inf), grad_q=z(q.shape),
             grad_k=z(k.shape), grad_v=z(v.shape), grad_slope=z(heads), grad_pos=z((q.shape[0], 3)),
             grad_key_pos=z((k.shape[0], 3)))
    o.update({"abs_" + n: z(t.shape) for n, t in o.items() if n != "lse"})
    for g in range(len(offsets) - 1):
        a, b = slice(offsets[g], offsets[g + 1]), slice(ko[g], ko[g + 1])
        if a.stop <= a.start or b.stop <= b.start:
            continue
        for h in range(heads):
            qh, kh, vh = q[a][:, cq[h]], k[b][:, cq[h]], v[b][:, cv[h]]
            s, th, d = scores(qh, kh, scale, cap, None if slope is None else slope[h], None if pos is None else pos[a],
                              None if kp is None else kp[b])
            top = s.max(1, keepdims=True)
            e = np.exp(s - top)
            p = e / e.sum(1, keepdims=True)
            rows = np.arange(a.start, a.stop)
            o["lse"][h, a] = ((top + np.log(e.sum(1, keepdims=True))) / np.log(2.0))[:, 0]
            o["out"][rows[:, None], cv[h]] = p @ vh
            o["abs_out"][rows[:, None], cv[h]] = p @ np.abs(vh)
            if grad_out is None:
                continue
            cols = np.arange(b.start, b.stop)
            go = grad_out[a][:, cv[h]]
            dp = go @ vh.T
            delta = (p * dp).sum(1, keepdims=True)
            ds = p * (dp - delta)
            mag = p * (np.abs(go) @ np.abs(vh).T + (p * (np.abs(go) @ np.abs(vh).T)).sum(1, keepdims=True))
            o["grad_v"][cols[:, None], cv[h]] = p.T @ go
            o["abs_grad_v"][cols[:, None], cv[h]] = p.T @ np.abs(go)
            if slope is not None:
                o["grad_slope"][h] -= (ds * d).sum()
                o["abs_grad_slope"][h] += (mag * d).sum()
                w = np.divide(-slope[h] * ds, d, out=np.zeros_like(ds), where=d > 0)
                wm = np.divide(np.abs(slope[h]) * mag, d, out=np.zeros_like(ds), where=d > 0)
                diff = pos[a][:, None] - kp[b][None]
                qn, kn = ("grad_pos", "grad_key_pos" if cross else "grad_pos")
                o[qn][a] += (w[..., None] * diff).sum(1)
                o[kn][b] -= (w[..., None] * diff).sum(0)
                o["abs_" + qn][a] += (wm[..., None] * np.abs(diff)).sum(1)
                o["abs_" + kn][b] += (wm[..., None] * np.abs(diff)).sum(0)
            if cap > 0:
                ds = ds * (1 - th * th)  # (the bounds keep the factor's largest value, 1)
            o["grad_q"][rows[:, None], cq[h]] = scale * (ds @ kh)
            o["grad_k"][cols[:, None], cq[h]] = scale * (ds.T @ qh)
            o["abs_grad_q"][rows[:, None], cq[h]] = abs(scale) * (mag @ np.abs(kh))
            o["abs_grad_k"][cols[:, None], cq[h]] = abs(scale) * (mag.T @ np.abs(qh))
    return o


def embed(index, W, scale):
    there = (index >= 0) & (index < W.shape[0])
    return np.where(there[:, None], scale * W[np.where(there, index, 0)], 0.0)


def embed_backward(index, grad_y, rows, scale):
    """(grad_W, the sums of the magnitudes)"""
    there = (index >= 0) & (index < rows)
    g, m = np.zeros((rows, grad_y.shape[1])), np.zeros((rows, grad_y.shape[1]))
    np.add.at(g, index[there], grad_y[there])
    np.add.at(m, index[there], np.abs(grad_y[there]))
    return scale * g, abs(scale) * m


def philox4x32(counter, key, rounds=10):
    """Philox4x32 (J. Salmon et al., 2011): counter [..., 4] and key [2] of 32-bit words."""
    c = [int(w) for w in counter]
    k = [int(w) for w in key]
    for _ in range(rounds):
        p0, p1 = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(p1 >> 32) ^ c[1] ^ k[0], p1 & 0xFFFFFFFF, (p0 >> 32) ^ c[3] ^ k[1], p0 & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def dropout_factors(text, nodes, p, seed, offset, first_node=0):
    """What every value of a node tensor is multiplied by: 0 or 65536 / (65536 - round(65536 p))."""
    blocks, F = irreps(text)
    limit = int(np.rint(np.float64(np.float32(p)) * 65536))
    keep = 65536.0 / (65536 - limit) if limit < 65536 else 0.0
    U = sum((b[0] + 7) // 8 for b in blocks)
    seed, offset = seed % (1 << 64), offset % (1 << 64)
    out = np.zeros((nodes, F))
    for v in range(nodes):
        u = 0
        for mul, n, _, at in blocks:
            for c in range(mul):
                b = (v + first_node) * U + u + c // 8
                w = philox4x32([b & 0xFFFFFFFF, b >> 32, offset & 0xFFFFFFFF, offset >> 32],
                               [seed & 0xFFFFFFFF, seed >> 32])[(c % 8) // 2]
                word = (w >> (16 * (c % 2))) & 0xFFFF
                out[v, at + c:at + mul * n:mul] = keep if word >= limit else 0.0
            u += (mul + 7) // 8
    return out
