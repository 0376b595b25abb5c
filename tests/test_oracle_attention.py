"""Pins of the attention block's fp64 definitions: closed forms, invariances, published generator values, differences."""
import numpy as np
import pytest

from oracle import attention as oa
from oracle import sh
from oracle.layers import irreps


def data(text_qk, text_v, lens, seed, key_lens=None):
    rng = np.random.default_rng(seed)
    nq, nk = sum(lens), sum(key_lens or lens)
    off = np.concatenate([[0], np.cumsum(lens)])
    ko = None if key_lens is None else np.concatenate([[0], np.cumsum(key_lens)])
    d = dict(q=rng.standard_normal((nq, irreps(text_qk)[1])), k=rng.standard_normal((nk, irreps(text_qk)[1])),
             v=rng.standard_normal((nk, irreps(text_v)[1])), offsets=off, key_offsets=ko, pos=rng.standard_normal((nq, 3)),
             key_pos=None if ko is None else rng.standard_normal((nk, 3)))
    return d, rng.standard_normal((nq, irreps(text_v)[1]))


def test_uniform_scores_give_means():
    d, _ = data("4x0e", "2x0e+2x1o", (3, 5), 0)
    d["q"] = np.zeros_like(d["q"])
    out = oa.attention("4x0e", "2x0e+2x1o", 2, **{n: d[n] for n in ("q", "k", "v", "offsets")})["out"]
    assert np.allclose(out[:3], d["v"][:3].mean(0)) and np.allclose(out[3:], d["v"][3:].mean(0))


def test_no_keys_give_zeros_and_one_key_its_value():
    d, g = data("4x0e", "4x0e", (2, 3), 1, (0, 1))
    o = oa.attention("4x0e", "4x0e", 1, d["q"], d["k"], d["v"], d["offsets"], d["key_offsets"], grad_out=g)
    assert np.all(o["out"][:2] == 0) and np.allclose(o["out"][2:], d["v"][0]) and np.all(o["lse"][0, :2] == -np.inf)
    assert np.allclose(o["grad_v"][0], g[2:].sum(0)) and np.allclose(o["grad_q"], 0) and np.allclose(o["grad_k"], 0)


def test_slopes_and_caps_limit():
    d, _ = data("4x0e", "4x0e", (6,), 2)
    base = dict(q=d["q"], k=d["k"], v=d["v"], offsets=d["offsets"], pos=d["pos"], scale=0.5)
    near = oa.attention("4x0e", "4x0e", 1, slope=np.array([1e4]), **base)["out"]
    assert np.allclose(near, d["v"])  # only itself is in the same place
    plain = oa.attention("4x0e", "4x0e", 1, **base)["out"]
    assert np.allclose(oa.attention("4x0e", "4x0e", 1, cap=1e6, **base)["out"], plain)
    assert np.allclose(oa.attention("4x0e", "4x0e", 1, cap=1e-9, **base)["out"], d["v"].mean(0))


def test_rotations_turn_the_outputs():
    text, heads = "4x0e+4x1o+2x2e", 2
    d, _ = data(text, text, (7,), 3)
    R = np.linalg.qr(np.random.default_rng(4).standard_normal((3, 3)))[0]
    R *= np.sign(np.linalg.det(R))

    def turn(x):
        out = x.copy()
        for mul, n, kind, at in irreps(text)[0]:
            l = (n - 1) // 2
            pts = np.random.default_rng(5).standard_normal((4 * n, 3))
            pts /= np.linalg.norm(pts, axis=1, keepdims=True)
            D = np.linalg.lstsq(sh.sh_single_l(l, pts), sh.sh_single_l(l, pts @ R.T), rcond=None)[0].T
            out[:, at:at + n * mul] = np.einsum("mn,vnc->vmc", D, x[:, at:at + n * mul].reshape(-1, n, mul)).reshape(
                -1, n * mul)
        return out

    args = dict(offsets=d["offsets"], slope=np.array([0.3, 0.1]), scale=0.2)
    a = oa.attention(text, text, heads, d["q"], d["k"], d["v"], pos=d["pos"], **args)["out"]
    b = oa.attention(text, text, heads, turn(d["q"]), turn(d["k"]), turn(d["v"]), pos=d["pos"] @ R.T + 5.0, **args)["out"]
    assert np.allclose(turn(a), b, atol=1e-10)


@pytest.mark.parametrize("cap,bias,key_lens", [(0.0, False, None), (2.0, True, None), (0.0, True, (3, 0, 4)),
                                               (1.5, False, (1, 2, 5))])
def test_gradients_against_differences(cap, bias, key_lens):
    qk, vv, heads, lens = "2x0e+2x1o", "4x0e+2x1o", 2, (3, 2, 4)
    d, g = data(qk, vv, lens, 6, key_lens)
    slope = np.array([0.7, 0.2]) if bias else None
    names = ["q", "k", "v"] + (["slope", "pos"] + (["key_pos"] if key_lens else []) if bias else [])

    def value(**new):
        a = dict(d, slope=slope, **{})
        a.update(new)
        if not bias:
            a["pos"] = a["key_pos"] = None
        return a

    def loss(a):
        return (oa.attention(qk, vv, heads, scale=0.4, cap=cap, **a)["out"] * g).sum()

    got = oa.attention(qk, vv, heads, scale=0.4, cap=cap, grad_out=g, **value())
    rng = np.random.default_rng(7)
    for n in names:
        base = slope if n == "slope" else d[n]
        for _ in range(4):
            u = rng.standard_normal(base.shape)
            h = 1e-6
            num = (loss(value(**{n: base + h * u})) - loss(value(**{n: base - h * u}))) / (2 * h)
            assert abs(num - (got["grad_" + n] * u).sum()) < 1e-6 * max(1.0, np.abs(got["grad_" + n]).sum())


def test_embedding_and_its_gradient_are_adjoint():
    rng = np.random.default_rng(8)
    z = np.array([0, 3, 3, -1, 7, 2, 0, 5])
    W, g = rng.standard_normal((5, 6)), rng.standard_normal((8, 6))
    y = oa.embed(z, W, 1.7)
    assert np.all(y[[3, 4, 7]] == 0) and np.allclose(y[1], 1.7 * W[3])
    gW, m = oa.embed_backward(z, g, 5, 1.7)
    assert np.isclose((y * g).sum(), (W * gW).sum()) and np.all(gW[[1, 4]] == 0) and np.all(np.abs(gW) <= m + 1e-15)


def test_philox_known_answers():
    """The generator's published known answers (Random123 1.x, philox4x32 with 10 rounds)."""
    f = 0xFFFFFFFF
    assert oa.philox4x32([0] * 4, [0] * 2) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert oa.philox4x32([f] * 4, [f] * 2) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    assert oa.philox4x32([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0]) == [
        0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]


def test_dropout_masks():
    text = "9x0e+5x1o+8x2e"
    f = oa.dropout_factors(text, 40, 0.25, -5, 1 << 40)
    assert set(np.unique(f)) == {0.0, 65536.0 / 49152.0}
    rows = f[:, 9:24].reshape(40, 3, 5)
    assert np.all(rows == rows[:, :1])  # shared by the rows of an irrep
    assert abs((f > 0).mean() - 0.75) < 0.06
    assert np.all(oa.dropout_factors(text, 3, 1.0, 1, 1) == 0) and np.all(oa.dropout_factors(text, 3, 0.0, 1, 1) == 1)
    again = oa.dropout_factors(text, 7, 0.25, -5, 1 << 40, first_node=33)
    assert np.all(again == f[33:]) and not np.all(f == oa.dropout_factors(text, 40, 0.25, -5, (1 << 40) + 1))
