"""Host side of the attention block's operators: exports, sizes and refusals (no GPU)."""
import ctypes
import os
import re
from ctypes import byref

import pytest
import torch

from equivariant_gnn_tensor_receiver_amd import tpconv as tp
from oracle.layers import irreps

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytestmark = pytest.mark.skipif(not os.path.exists(tp.LIB_PATH), reason="libtpconv.so not built")
if os.path.exists(tp.LIB_PATH):
    from equivariant_gnn_tensor_receiver_amd import attention as at
    from equivariant_gnn_tensor_receiver_amd import layers as ly

FAKE, BIG = ctypes.c_void_p(64).value, 1 << 40


def test_exports_every_declared_symbol():
    text = open(os.path.join(ROOT, "include", "tpconv_attention.h")).read()
    names = sorted(set(re.findall(r"^tpconv_status\s+(tpconv_\w+)\s*\(", text, re.M)))
    assert names == sorted(at.EXPORTS)
    for n in names:
        assert hasattr(ctypes.CDLL(tp.LIB_PATH), n), n
    for name in re.findall(r"TPCONV_KERNEL_(\w+) = (\d+)", text):
        assert tp.KERNELS[int(name[1])] == name[0].lower()
    count = int(re.search(r"TPCONV_KERNEL_COUNT = (\d+)", open(os.path.join(ROOT, "include", "tpconv.h")).read())[1])
    assert len(tp.KERNELS) == count


def status(make):
    with pytest.raises(tp.TpconvError) as e:
        make()
    return e.value.status


def test_refused_descriptors():
    assert status(lambda: at.Attention("8x0q", "8x0e", 2)) == 2
    assert status(lambda: at.Attention("8x0e", "", 2)) == 2
    assert status(lambda: at.Attention("8x0e+3x1o", "8x0e", 2)) == 2  # channels that do not divide
    assert status(lambda: at.Attention("8x0e", "7x0e", 2)) == 2
    assert status(lambda: at.Attention("8x4e", "8x0e", 2)) == 5
    assert status(lambda: at.Attention("8x0e", "+".join(["2x0e"] * 17), 2)) == 5
    assert status(lambda: at.Attention("514x0e", "8x0e", 2)) == 5  # 257 values per head
    assert status(lambda: at.Attention("8x0e", "64x0e+64x1o+64x2e", 2)) == 5
    for heads in (0, -1, 257):
        assert status(lambda: at.Attention("8x0e", "8x0e", heads)) == 1
    for scale, cap in ((float("nan"), 0.0), (float("inf"), 0.0), (1.0, -1.0), (1.0, float("nan")), (1.0, float("inf"))):
        assert status(lambda: at.Attention("8x0e", "8x0e", 2, scale, cap)) == 1
    assert status(lambda: at.Attention("8x0e", "8x0e", 2, x_dtype=2)) == 1
    assert status(lambda: at.Attention("8x0e", "8x0e", 2, y_dtype=-1)) == 1
    for rows, f, scale in ((0, 4, 1.0), (-1, 4, 1.0), (2 ** 24 + 1, 4, 1.0), (4, 0, 1.0), (4, 65537, 1.0),
                           (4, 4, float("nan")), (4, 4, float("inf"))):
        assert status(lambda: at.Embedding(rows, f, scale)) == 1
    assert status(lambda: at.Embedding(4, 4, 1.0, 3)) == 1
    for p in (-0.1, 1.1, float("nan")):
        assert status(lambda: at.Dropout("8x0e", p)) == 1
    assert status(lambda: at.Dropout("8x0", 0.1)) == 2
    assert status(lambda: at.Dropout("8x4e", 0.1)) == 5
    assert status(lambda: at.Dropout("8x0e", 0.1, 0, 5)) == 1


def test_refused_scales_and_caps():
    """What the kernels would make of them (scale / cap, 1 / cap, both times log2(e)) has to be in fp32's range."""
    for scale, cap in ((2.0 ** 101, 0.0), (-2.0 ** 101, 0.0), (1.0, 2.0 ** -101), (1.0, 2.0 ** 101), (2.0 ** 100, 2.0 ** -100),
                       (1.0, 1e-45)):
        assert status(lambda: at.Attention("8x0e", "8x0e", 2, scale, cap)) == 1
    for scale, cap in ((2.0 ** 100, 0.0), (-1.0, 0.0), (0.0, 1.0), (1.0, 2.0 ** -100), (1.0, 2.0 ** 100)):
        assert at.Attention("8x0e", "8x0e", 2, scale, cap).scale == scale


def test_a_batch_notices_replaced_memory():
    off, pos = torch.tensor([0, 2, 5], dtype=torch.int32), torch.zeros(5, 3)
    b = at.Batch(5, off, pos)
    b.check()
    pos[0] = 1.0  # new values are fine
    b.check()
    pos.data = torch.zeros(5, 3)
    with pytest.raises(ValueError, match="other memory"):
        b.check()
    b = at.Batch(5, off)
    off.data = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="other memory"):
        b.check()


def test_sizes():
    h = at.Attention("16x0e+8x1o", "32x0e+8x2e", 8)
    assert (h.feat_qk, h.feat_v, h.head_qk, h.head_v) == (irreps("16x0e+8x1o")[1], irreps("32x0e+8x2e")[1], 5, 9)
    assert h.scale == 5 ** -0.5
    assert h.saved_size(10) == 160 and at.Attention("8x0e", "8x0e", 2, y_dtype=at.TPCONV_BF16).saved_size(10) == 120
    assert at.Attention("256x0e", "256x0e", 1).head_qk == 256
    few = at.Batch(4096, torch.zeros(129, dtype=torch.int32))
    assert h.workspace_size(few, at.OP_FORWARD) == 0 and h.workspace_size(few) > 0
    one = at.Batch(1, torch.zeros(2, dtype=torch.int32), None, 100000, torch.zeros(2, dtype=torch.int32))
    assert h.workspace_size(one, at.OP_FORWARD) > 0  # one query, many keys: cut into parts
    assert at.Embedding(10, 8).workspace_size(64) == 0 and at.Embedding(10, 8).workspace_size(5000) > 0
    assert at.Dropout("8x0e+2x1o", 0.25).features == 14 and at.Dropout("1x0e", 0.25).p == 0.25


def batch(**kw):
    b = dict(num_graphs=2, num_queries=4, offsets=FAKE, pos=None, num_keys=0, key_offsets=None, key_pos=None)
    return at.AttentionBatch(*dict(b, **kw).values())


def inputs(**kw):
    i = dict(q=FAKE, k=FAKE, v=FAKE, q_stride=0, k_stride=0, v_stride=0, slope=None)
    return at.AttentionInputs(*dict(i, **kw).values())


def grads(**kw):
    g = dict(grad_q=None, grad_k=None, grad_v=None, q_stride=0, k_stride=0, v_stride=0, grad_slope=None, grad_pos=None,
             grad_key_pos=None)
    return at.AttentionGrads(*dict(g, **kw).values())


def test_refused_arguments_before_any_launch():
    L = at._lib()
    a = at.Attention("8x0e", "8x0e", 2)
    h = a.handle

    def forward(b=batch(), i=inputs(), out=FAKE, ws=FAKE, size=BIG, handle=h):
        return L.tpconv_attention_forward(handle, None if b is None else byref(b), None if i is None else byref(i), out,
                                          None, ws, size, None)

    assert forward(handle=None) == 1 and forward(b=None) == 1 and forward(i=None) == 1 and forward(out=None) == 1
    for kw in (dict(num_queries=-1), dict(num_queries=2 ** 31), dict(num_graphs=-1), dict(offsets=None),
               dict(key_offsets=FAKE, num_keys=-1), dict(offsets=None, num_graphs=1, key_offsets=FAKE, num_keys=4)):
        assert forward(batch(**kw)) == 1, kw
    for kw in (dict(q=None), dict(k=None), dict(v=None), dict(q_stride=7), dict(k_stride=-8), dict(v_stride=7),
               dict(slope=FAKE)):  # slopes without positions
        assert forward(i=inputs(**kw)) == 1, kw
    assert forward(batch(key_offsets=FAKE, num_keys=4, pos=FAKE), inputs(slope=FAKE)) == 1
    assert forward(batch(num_queries=0), inputs(q=None, k=None, v=None)) == 0
    parts = batch(num_graphs=1, num_queries=1, key_offsets=FAKE, num_keys=100000)
    size = ctypes.c_size_t()
    assert L.tpconv_attention_workspace_size(h, at.OP_FORWARD, byref(parts), byref(size)) == 0 and size.value > 0
    assert forward(parts, ws=None) == 4 and forward(parts, size=size.value - 1) == 4 and forward(parts, ws=FAKE + 8) == 4
    assert L.tpconv_attention_workspace_size(h, tp.OP_DOUBLE_BACKWARD, byref(parts), byref(size)) == 1
    huge = batch(num_graphs=2 ** 30, num_queries=2 ** 30)
    assert L.tpconv_attention_workspace_size(h, at.OP_FORWARD, byref(huge), byref(size)) == 5

    def backward(g, b=batch(pos=FAKE), i=inputs(slope=FAKE), out=FAKE, saved=FAKE, go=FAKE, ws=FAKE, size=BIG):
        return L.tpconv_attention_backward(h, byref(b), byref(i), out, saved, go, None if g is None else byref(g), ws,
                                           size, None)

    every = dict(grad_q=FAKE, grad_k=FAKE, grad_v=FAKE, grad_slope=FAKE, grad_pos=FAKE)
    assert backward(None) == 1 and backward(grads()) == 1
    assert backward(grads(**every, grad_key_pos=FAKE)) == 1  # self form
    assert backward(grads(grad_slope=FAKE), i=inputs()) == 1 and backward(grads(grad_pos=FAKE), i=inputs()) == 1
    for kw in (dict(q_stride=3), dict(k_stride=-1), dict(v_stride=7)):
        assert backward(grads(**dict(every, **kw))) == 1
    for kw in (dict(out=None), dict(saved=None), dict(go=None)):
        assert backward(grads(**every), **kw) == 1
    need = ctypes.c_size_t()
    assert L.tpconv_attention_workspace_size(h, at.OP_BACKWARD, byref(batch(pos=FAKE)), byref(need)) == 0
    assert backward(grads(**every), size=need.value - 1) == 4 and backward(grads(**every), ws=FAKE + 4) == 4

    e = at.Embedding(5, 4)
    n = e.workspace_size(200)
    assert L.tpconv_embed_forward(None, 4, FAKE, FAKE, FAKE, None) == 1
    assert L.tpconv_embed_forward(e.handle, -1, FAKE, FAKE, FAKE, None) == 1
    for k in range(3):
        assert L.tpconv_embed_forward(e.handle, 4, *[None if j == k else FAKE for j in range(3)], None) == 1
        assert L.tpconv_embed_backward(e.handle, 200, *[None if j == k else FAKE for j in range(3)], FAKE, BIG, None) == 1
    assert L.tpconv_embed_forward(e.handle, 0, None, None, None, None) == 0
    assert L.tpconv_embed_backward(e.handle, 200, FAKE, FAKE, FAKE, FAKE, n - 1, None) == 4
    assert L.tpconv_embed_backward(e.handle, 200, FAKE, FAKE, FAKE, None, n, None) == 4
    assert L.tpconv_embed_backward(e.handle, 200, FAKE, FAKE, FAKE, FAKE + 8, n, None) == 4

    d = at.Dropout("8x0e", 0.5, 0, 1)
    assert L.tpconv_dropout_forward(None, 4, FAKE, FAKE, None, FAKE, None) == 1
    assert L.tpconv_dropout_forward(d.handle, -4, FAKE, FAKE, None, FAKE, None) == 1
    assert L.tpconv_dropout_forward(d.handle, 4, FAKE, FAKE, None, FAKE, None) == 1  # in place, but types differ
    for k in range(3):
        args = [None if j == k else v for j, v in enumerate((FAKE, FAKE, FAKE + 64))]
        assert L.tpconv_dropout_forward(d.handle, 4, args[0], args[1], None, args[2], None) == 1
        assert L.tpconv_dropout_backward(d.handle, 4, *args, None) == 1
    assert L.tpconv_dropout_forward(d.handle, 0, None, None, None, None, None) == 0


@pytest.fixture
def calls(monkeypatch):
    """CPU tensors in place of device tensors; the names of the library calls that would be made."""
    made = []
    monkeypatch.setattr(ly, "_device", lambda t, name: t.device)
    monkeypatch.setattr(ly, "_call", lambda fn, device, stream, *args: made.append(fn))
    return made


def test_binding_refuses_tensors_the_kernels_would_misread(calls):
    h, b = at.Attention("8x0e", "6x0e", 2), at.Batch(3)
    q, v = torch.zeros(3, 8), torch.zeros(3, 6)
    assert at.tpconv_attention_forward(h, b, q, q, v).shape == (3, 6)
    wide = torch.zeros(3, 30)
    at.tpconv_attention_forward(h, b, wide[:, :8], wide[:, 8:16], wide[:, 16:22])
    made = len(calls)
    bad = [torch.zeros(3, 7), torch.zeros(2, 8), torch.zeros(3, 8, dtype=torch.bfloat16), torch.zeros(8, 3).t(),
           torch.zeros(3, 16)[:, ::2], torch.zeros(1, 8).expand(3, 8), torch.zeros(3, 8, dtype=torch.float64)]
    for t in bad:
        for args in ((t, q, v), (q, t, v)):
            with pytest.raises((ValueError, TypeError)):
                at.tpconv_attention_forward(h, b, *args)
    with pytest.raises(ValueError, match="positions"):
        at.tpconv_attention_forward(h, b, q, q, v, slope=torch.ones(2))
    with pytest.raises(ValueError, match="slope"):
        at.tpconv_attention_forward(h, at.Batch(3, pos=torch.zeros(3, 3)), q, q, v, slope=torch.ones(3))
    saved = torch.zeros(h.saved_size(3))
    for want, kw in ((("slope",), {}), (("pos",), {}), ((), dict(grad_key_pos=torch.zeros(3, 3))),
                     ((), dict(grad_q=torch.zeros(3, 9))), ((), dict(grad_q=torch.zeros(1, 8).expand(3, 8)))):
        with pytest.raises((ValueError, TypeError)):
            at.tpconv_attention_backward(h, b, q, q, v, v, saved, v, want=want, **kw)
    with pytest.raises(ValueError, match="saved"):
        at.tpconv_attention_backward(h, b, q, q, v, v, saved[1:], v)
    off = torch.zeros(3, dtype=torch.int32)
    for kw in (dict(num_keys=4), dict(key_pos=torch.zeros(3, 3)), dict(key_offsets=off, num_keys=4),
               dict(offsets=off, key_offsets=off), dict(offsets=off, key_offsets=off[:2], num_keys=4),
               dict(pos=torch.zeros(4, 3)), dict(offsets=off[::2]),
               dict(offsets=off, key_offsets=off, num_keys=4, key_pos=torch.zeros(3, 3))):
        with pytest.raises(ValueError):
            at.Batch(3, **kw)
    for kw in (dict(offsets=off.long()), dict(pos=torch.zeros(3, 3, dtype=torch.float64))):
        with pytest.raises(TypeError):
            at.Batch(3, **kw)
    e, z = at.Embedding(5, 4), torch.zeros(3, dtype=torch.int32)
    for index, W in ((z.long(), torch.zeros(5, 4)), (z, torch.zeros(4, 4)), (z, torch.zeros(5, 4).bfloat16())):
        with pytest.raises((ValueError, TypeError)):
            at.tpconv_embed_forward(e, index, W)
    d, x = at.Dropout("3x1o", 0.5), torch.zeros(2, 9)
    rng = torch.zeros(2, dtype=torch.int64)
    for args, kw in (((x, rng[:1]), {}), ((x, rng.int()), {}), ((torch.zeros(2, 8), rng), {}),
                     ((x, rng), dict(residual=torch.zeros(1, 9))), ((x, rng), dict(out=x.bfloat16()))):
        with pytest.raises((ValueError, TypeError)):
            at.tpconv_dropout_forward(d, *args, **kw)
    assert len(calls) == made


def test_binding_needs_a_gpu():
    with pytest.raises(ValueError, match="GPU"):
        at.tpconv_dropout_forward(at.Dropout("1x0e", 0.5), torch.zeros(1), torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="GPU"):
        at.tpconv_embed_forward(at.Embedding(2, 2), torch.zeros(1, dtype=torch.int32), torch.zeros(2, 2))
    with pytest.raises(ValueError, match="GPU"):
        at.tpconv_attention_forward(at.Attention("1x0e", "1x0e", 1), at.Batch(1), *[torch.zeros(1, 1)] * 3)
