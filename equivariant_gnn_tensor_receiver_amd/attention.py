"""Python binding of the attention block's operators (the C ABI in include/tpconv_attention.h): attention among the
nodes of each graph of a batch, the embedding of node types, and dropout from a counter-based generator.

As in ``layers``: argument marshalling only, functions carry the C names, PyTorch provides device memory and the current
HIP stream.  Tensors are contiguous, except that q, k, v and their gradients may be column ranges [N][F] of a wider
tensor (rows of any stride).
"""
from __future__ import annotations

import ctypes
from ctypes import POINTER, byref, c_char_p, c_float, c_int32, c_int64, c_size_t, c_void_p

import torch

from . import layers as ly
from . import tpconv as tp
from .tpconv import OP_BACKWARD, OP_FORWARD, TPCONV_BF16, TPCONV_F32  # noqa: F401  (part of this module's interface)

EXPORTS = ("tpconv_attention_create", "tpconv_attention_destroy", "tpconv_attention_info",
           "tpconv_attention_saved_size", "tpconv_attention_workspace_size", "tpconv_attention_forward",
           "tpconv_attention_backward", "tpconv_embed_create", "tpconv_embed_destroy", "tpconv_embed_workspace_size",
           "tpconv_embed_forward", "tpconv_embed_backward", "tpconv_dropout_create", "tpconv_dropout_destroy",
           "tpconv_dropout_info", "tpconv_dropout_forward", "tpconv_dropout_backward")


class AttentionDesc(ctypes.Structure):
    _fields_ = [("irreps_qk", c_char_p), ("irreps_v", c_char_p), ("num_heads", c_int32), ("scale", c_float),
                ("score_cap", c_float), ("x_dtype", c_int32), ("y_dtype", c_int32)]


class AttentionBatch(ctypes.Structure):
    _fields_ = [("num_graphs", c_int64), ("num_queries", c_int64), ("offsets", c_void_p), ("pos", c_void_p),
                ("num_keys", c_int64), ("key_offsets", c_void_p), ("key_pos", c_void_p)]


class AttentionInputs(ctypes.Structure):
    _fields_ = [("q", c_void_p), ("k", c_void_p), ("v", c_void_p), ("q_stride", c_int64), ("k_stride", c_int64),
                ("v_stride", c_int64), ("slope", c_void_p)]


class AttentionGrads(ctypes.Structure):
    _fields_ = [("grad_q", c_void_p), ("grad_k", c_void_p), ("grad_v", c_void_p), ("q_stride", c_int64),
                ("k_stride", c_int64), ("v_stride", c_int64), ("grad_slope", c_void_p), ("grad_pos", c_void_p),
                ("grad_key_pos", c_void_p)]


class EmbedDesc(ctypes.Structure):
    _fields_ = [("num_rows", c_int32), ("features", c_int32), ("scale", c_float), ("w_dtype", c_int32),
                ("y_dtype", c_int32)]


class DropoutDesc(ctypes.Structure):
    _fields_ = [("irreps", c_char_p), ("p", c_float), ("x_dtype", c_int32), ("y_dtype", c_int32)]


_LIB = None


def _lib():
    global _LIB
    if _LIB is None:
        L = ly._lib()
        P, N, I, S = c_void_p, c_int64, c_int32, c_size_t
        L.tpconv_attention_create.argtypes = [POINTER(P), POINTER(AttentionDesc)]
        L.tpconv_attention_destroy.argtypes = [P]
        L.tpconv_attention_info.argtypes = [P, POINTER(N), POINTER(N), POINTER(I), POINTER(I)]
        L.tpconv_attention_saved_size.argtypes = [P, N, POINTER(N)]
        L.tpconv_attention_workspace_size.argtypes = [P, I, P, POINTER(S)]
        L.tpconv_attention_forward.argtypes = [P, P, P, P, P, P, S, P]
        L.tpconv_attention_backward.argtypes = [P, P, P, P, P, P, P, P, S, P]
        L.tpconv_embed_create.argtypes = [POINTER(P), POINTER(EmbedDesc)]
        L.tpconv_embed_destroy.argtypes = [P]
        L.tpconv_embed_workspace_size.argtypes = [P, N, POINTER(S)]
        L.tpconv_embed_forward.argtypes = [P, N, P, P, P, P]
        L.tpconv_embed_backward.argtypes = [P, N, P, P, P, P, S, P]
        L.tpconv_dropout_create.argtypes = [POINTER(P), POINTER(DropoutDesc)]
        L.tpconv_dropout_destroy.argtypes = [P]
        L.tpconv_dropout_info.argtypes = [P, POINTER(N), POINTER(c_float)]
        L.tpconv_dropout_forward.argtypes = [P, N, P, P, P, P, P]
        L.tpconv_dropout_backward.argtypes = [P, N, P, P, P, P]
        for name in EXPORTS:
            getattr(L, name).restype = I
        _LIB = L
    return _LIB


# ---- attention ------------------------------------------------------------------------


class Attention(ly._Handle):
    """Attention among the nodes of each graph, on irreps features with num_heads heads.  scale: of the scores, by
    default one over the square root of the values per head; score_cap > 0: scores s become cap tanh(s / cap)."""

    _destroy = "tpconv_attention_destroy"

    def __init__(self, irreps_qk: str, irreps_v: str, num_heads: int, scale: float | None = None,
                 score_cap: float = 0.0, x_dtype: int = TPCONV_F32, y_dtype: int = TPCONV_F32):
        L, h = _lib(), c_void_p()

        def create(scale):
            desc = AttentionDesc(irreps_qk.encode(), irreps_v.encode(), num_heads, scale, score_cap, x_dtype, y_dtype)
            tp._check(L.tpconv_attention_create(byref(h), byref(desc)), "tpconv_attention_create")
            fq, fv, dq, dv = c_int64(), c_int64(), c_int32(), c_int32()
            tp._check(L.tpconv_attention_info(h, *(byref(v) for v in (fq, fv, dq, dv))), "tpconv_attention_info")
            return fq.value, fv.value, dq.value, dv.value

        got = create(1.0 if scale is None else scale)
        if scale is None:
            L.tpconv_attention_destroy(h)
            scale = got[2] ** -0.5
            got = create(scale)
        self.handle = h
        self.feat_qk, self.feat_v, self.head_qk, self.head_v = got
        self.num_heads, self.scale, self.score_cap = num_heads, scale, score_cap
        self.x_dtype, self.y_dtype = ly._dtype(x_dtype), ly._dtype(y_dtype)
        self._ws = {}

    def saved_size(self, num_queries: int) -> int:
        """fp32 values a forward saves for its backward."""
        n = c_int64()
        tp._check(_LIB.tpconv_attention_saved_size(self.handle, num_queries, byref(n)), "tpconv_attention_saved_size")
        return n.value

    def workspace_size(self, batch: "Batch", op: int = OP_BACKWARD) -> int:
        key = (batch.key, op)
        size = self._ws.get(key)  # other threads may ask the same handle, and replace the dict
        if size is None:
            b = c_size_t()
            tp._check(_LIB.tpconv_attention_workspace_size(self.handle, op, batch.ref, byref(b)),
                      "tpconv_attention_workspace_size")
            size = b.value
            if len(self._ws) > 16:
                self._ws = {}
            self._ws[key] = size
        return size


def _whole(t, name, dtype, numel, device):
    if t is not None:
        ly._need(t, name, dtype, numel, device)


class Batch:
    """Which rows belong to which graph: graph g's queries are the rows offsets[g] .. offsets[g + 1] - 1 (device int32;
    None: one graph of all rows), its keys the queries' own nodes, or with key_offsets rows of their own.  pos, key_pos:
    fp32 positions [rows][3] for the distance bias.  Not changed after it is made."""

    def __init__(self, num_queries: int, offsets=None, pos=None, num_keys: int | None = None, key_offsets=None,
                 key_pos=None):
        if key_offsets is None and (num_keys is not None or key_pos is not None):
            raise ValueError("key_offsets: needed for keys of their own")
        if key_offsets is not None and (num_keys is None or offsets is None):
            raise ValueError("num_keys, offsets: needed with key_offsets")
        self.num_queries, self.num_keys = num_queries, num_queries if key_offsets is None else num_keys
        self.offsets, self.pos, self.key_offsets, self.key_pos = offsets, pos, key_offsets, key_pos
        self.num_graphs = 1 if offsets is None else offsets.numel() - 1
        self.cross = key_offsets is not None
        for t in (offsets, pos, key_offsets, key_pos):
            if t is not None:
                dev = t.device
                _whole(offsets, "offsets", torch.int32, max(1, self.num_graphs + 1), dev)
                _whole(key_offsets, "key_offsets", torch.int32, self.num_graphs + 1, dev)
                _whole(pos, "pos", torch.float32, 3 * num_queries, dev)
                _whole(key_pos, "key_pos", torch.float32, 3 * self.num_keys, dev)
                self.device = dev
                break
        else:
            self.device = None
        self.struct = AttentionBatch(self.num_graphs, num_queries, ly._ptr(offsets), ly._ptr(pos), self.num_keys,
                                     ly._ptr(key_offsets), ly._ptr(key_pos))
        self.ref = byref(self.struct)
        self._made = tuple((t, t.data_ptr(), t.numel()) for t in (offsets, pos, key_offsets, key_pos) if t is not None)
        self.key = (self.num_graphs, num_queries, self.num_keys, self.cross, pos is not None, key_pos is not None)

    def check(self):
        """Raises if a tensor of the batch has since been given other memory (``.data``, ``set_``, ``resize_``)."""
        for t, at, numel in self._made:
            if t.data_ptr() != at or t.numel() != numel:
                raise ValueError("batch: a tensor of it has other memory than when it was made")


def _rows(t, name, dtype, n, features, device):
    """The row stride of n rows of `features` values: 0 for a contiguous tensor of any shape."""
    if t.dtype == dtype and t.device == device:
        if t.is_contiguous() and t.numel() == n * features:
            return 0
        if t.dim() == 2 and t.shape == (n, features) and t.stride(1) == 1 and t.stride(0) >= features:
            return t.stride(0)
    if t.dim() == 2 and t.shape == (n, features) and not t.is_contiguous():
        tp._require(t[:0], name, dtype, None, device)
        raise ValueError(f"{name}: rows must be contiguous and apart (strides {tuple(t.stride())})")
    tp._require(t, name, dtype, n * features, device)
    return 0


def _attention_inputs(attn, batch, q, k, v, slope, dev):
    if batch.device is not None and batch.device != dev:
        raise ValueError(f"batch: on {batch.device}, expected {dev}")
    batch.check()
    nq, nk = batch.num_queries, batch.num_keys
    s = (_rows(q, "q", attn.x_dtype, nq, attn.feat_qk, dev), _rows(k, "k", attn.x_dtype, nk, attn.feat_qk, dev),
         _rows(v, "v", attn.x_dtype, nk, attn.feat_v, dev))
    if slope is not None:
        ly._need(slope, "slope", torch.float32, attn.num_heads, dev)
        if (nq and batch.pos is None) or (batch.cross and nk and batch.key_pos is None):
            raise ValueError("slope: the batch has no positions")
    return AttentionInputs(q.data_ptr(), k.data_ptr(), v.data_ptr(), *s, ly._ptr(slope))


def tpconv_attention_forward(attn: Attention, batch: Batch, q, k, v, slope=None, out=None, saved=None, workspace=None,
                             stream=None):
    """out [num_queries][F_v].  slope: fp32 [num_heads], for the bias -slope |r_i - r_j| (needs the batch's positions).
    saved: fp32 tensor of attn.saved_size(num_queries) values for the backward.  Rows outside of all graphs are not
    written: in a result that the call makes they hold anything, so that padded batches, whose next layer runs over all
    rows, pass a cleared `out`."""
    dev = ly._device(q, "q")
    args = _attention_inputs(attn, batch, q, k, v, slope, dev)
    n = batch.num_queries
    if out is None:
        out = ly._new((n, attn.feat_v), attn.y_dtype, dev, stream)
    else:
        ly._need(out, "out", attn.y_dtype, n * attn.feat_v, dev)
    if saved is not None:
        ly._need(saved, "saved", torch.float32, attn.saved_size(n), dev)
    workspace, nbytes = ly._scratch(workspace, attn.workspace_size(batch, OP_FORWARD), dev, stream)
    ly._call("tpconv_attention_forward", dev, stream, attn.handle, batch.ref, byref(args), out.data_ptr(),
             ly._ptr(saved), ly._ptr(workspace), nbytes)
    return out


def tpconv_attention_backward(attn: Attention, batch: Batch, q, k, v, out, saved, grad_out, slope=None,
                              want=("q", "k", "v"), workspace=None, stream=None, grad_q=None, grad_k=None, grad_v=None,
                              grad_slope=None, grad_pos=None, grad_key_pos=None):
    """(grad_q, grad_k, grad_v, grad_slope, grad_pos, grad_key_pos) for the names in `want` ("q", "k", "v", "slope",
    "pos"), fp32; the others are None.  grad_pos is of the queries' positions, and in the self form of the nodes';
    grad_key_pos comes with "pos" in the cross form.  out, saved: of the forward on the same inputs.  Rows outside of
    all graphs are not written, in gradients that the call makes neither (padded batches pass cleared ones)."""
    dev = ly._device(q, "q")
    args = _attention_inputs(attn, batch, q, k, v, slope, dev)
    nq, nk, f32 = batch.num_queries, batch.num_keys, torch.float32
    ly._need(out, "out", attn.y_dtype, nq * attn.feat_v, dev)
    ly._need(saved, "saved", f32, attn.saved_size(nq), dev)
    ly._need(grad_out, "grad_out", f32, nq * attn.feat_v, dev)
    new = lambda *shape: ly._new(shape, f32, dev, stream)  # noqa: E731
    if grad_q is None and "q" in want:
        grad_q = new(nq, attn.feat_qk)
    if grad_k is None and "k" in want:
        grad_k = new(nk, attn.feat_qk)
    if grad_v is None and "v" in want:
        grad_v = new(nk, attn.feat_v)
    if grad_slope is None and "slope" in want:
        grad_slope = new(attn.num_heads)
    if "pos" in want:
        if grad_pos is None:
            grad_pos = new(nq, 3)
        if grad_key_pos is None and batch.cross:
            grad_key_pos = new(nk, 3)
    if slope is None and any(t is not None for t in (grad_slope, grad_pos, grad_key_pos)):
        raise ValueError("slope: needed for its gradient and those of the positions")
    if grad_key_pos is not None and not batch.cross:
        raise ValueError("grad_key_pos: the keys are the queries' nodes")
    strides = [0 if t is None else _rows(t, name, f32, n, f, dev) for t, name, n, f in
               ((grad_q, "grad_q", nq, attn.feat_qk), (grad_k, "grad_k", nk, attn.feat_qk),
                (grad_v, "grad_v", nk, attn.feat_v))]
    _whole(grad_slope, "grad_slope", f32, attn.num_heads, dev)
    _whole(grad_pos, "grad_pos", f32, 3 * nq, dev)
    _whole(grad_key_pos, "grad_key_pos", f32, 3 * nk, dev)
    got = (grad_q, grad_k, grad_v, grad_slope, grad_pos, grad_key_pos)
    if ly._nothing_to_compute(*got):
        return got
    workspace, nbytes = ly._scratch(workspace, attn.workspace_size(batch), dev, stream)
    p = [ly._ptr(t) for t in got]
    grads = AttentionGrads(*p[:3], *strides, *p[3:])
    ly._call("tpconv_attention_backward", dev, stream, attn.handle, batch.ref, byref(args), out.data_ptr(),
             saved.data_ptr(), grad_out.data_ptr(), byref(grads), ly._ptr(workspace), nbytes)
    return got


# ---- embedding ------------------------------------------------------------------------


class Embedding(ly._Handle):
    """scale * W[type], W [num_rows][features]; types outside of the table give zeros."""

    _destroy = "tpconv_embed_destroy"

    def __init__(self, num_rows: int, features: int, scale: float = 1.0, w_dtype: int = TPCONV_F32,
                 y_dtype: int = TPCONV_F32):
        L, h = _lib(), c_void_p()
        desc = EmbedDesc(num_rows, features, scale, w_dtype, y_dtype)
        tp._check(L.tpconv_embed_create(byref(h), byref(desc)), "tpconv_embed_create")
        self.handle = h
        self.num_rows, self.features, self.w_shape = num_rows, features, (num_rows, features)
        self.w_dtype, self.y_dtype = ly._dtype(w_dtype), ly._dtype(y_dtype)
        self._ws = (None, 0)

    def workspace_size(self, num_nodes: int) -> int:
        last, size = self._ws  # one read and one store: other threads may ask the same handle
        if last != num_nodes:
            b = c_size_t()
            tp._check(_LIB.tpconv_embed_workspace_size(self.handle, num_nodes, byref(b)), "tpconv_embed_workspace_size")
            size = b.value
            self._ws = (num_nodes, size)
        return size


def tpconv_embed_forward(embed: Embedding, index, W, out=None, stream=None):
    """y [N][features] for the types `index` (int32 [N])."""
    dev = ly._device(index, "index")
    n = index.numel()
    ly._need(index, "index", torch.int32, n, dev)
    ly._need(W, "W", embed.w_dtype, embed.num_rows * embed.features, dev)
    if out is None:
        out = ly._new((n, embed.features), embed.y_dtype, dev, stream)
    else:
        ly._need(out, "out", embed.y_dtype, n * embed.features, dev)
    ly._call("tpconv_embed_forward", dev, stream, embed.handle, n, index.data_ptr(), W.data_ptr(), out.data_ptr())
    return out


def tpconv_embed_backward(embed: Embedding, index, grad_y, grad_W=None, workspace=None, stream=None):
    """grad_W [num_rows][features], fp32; rows of types without nodes are zero."""
    dev = ly._device(index, "index")
    n = index.numel()
    ly._need(index, "index", torch.int32, n, dev)
    ly._need(grad_y, "grad_y", torch.float32, n * embed.features, dev)
    if grad_W is None:
        grad_W = ly._new(embed.w_shape, torch.float32, dev, stream)
    else:
        ly._need(grad_W, "grad_W", torch.float32, embed.num_rows * embed.features, dev)
    workspace, nbytes = ly._scratch(workspace, embed.workspace_size(n), dev, stream)
    ly._call("tpconv_embed_backward", dev, stream, embed.handle, n, index.data_ptr(), grad_y.data_ptr(),
             grad_W.data_ptr(), ly._ptr(workspace), nbytes)
    return grad_W


# ---- dropout --------------------------------------------------------------------------


class Dropout(ly._Handle):
    """Dropout of channels of a node tensor [N][F], the same for all rows of an irrep.  `p` is rounded to 16 bits."""

    _destroy = "tpconv_dropout_destroy"

    def __init__(self, irreps: str, p: float, x_dtype: int = TPCONV_F32, y_dtype: int = TPCONV_F32):
        L, h = _lib(), c_void_p()
        desc = DropoutDesc(irreps.encode(), p, x_dtype, y_dtype)
        tp._check(L.tpconv_dropout_create(byref(h), byref(desc)), "tpconv_dropout_create")
        self.handle = h
        f, used = c_int64(), c_float()
        tp._check(L.tpconv_dropout_info(h, byref(f), byref(used)), "tpconv_dropout_info")
        self.features, self.p = f.value, used.value
        self.x_dtype, self.y_dtype = ly._dtype(x_dtype), ly._dtype(y_dtype)


def _dropout_nodes(drop, t, name):
    n, rest = divmod(t.numel(), drop.features)
    if rest:
        raise ValueError(f"{name}: {t.numel()} elements, not a multiple of the {drop.features} features of a node")
    return n


def tpconv_dropout_forward(drop: Dropout, x, rng, residual=None, out=None, stream=None):
    """residual + dropout(x), in x's shape.  rng: int64 [2] = (seed, offset) on the device, read when the kernel runs;
    calls with the same values draw the same mask, so that every layer of every step needs an offset of its own.  out may be residual, or x if their types agree."""
    dev = ly._device(x, "x")
    n = _dropout_nodes(drop, x, "x")
    ly._need(x, "x", drop.x_dtype, n * drop.features, dev)
    ly._need(rng, "rng", torch.int64, 2, dev)
    if residual is not None:
        ly._need(residual, "residual", drop.y_dtype, n * drop.features, dev)
    if out is None:
        out = ly._new(x.shape, drop.y_dtype, dev, stream, x)
    else:
        ly._need(out, "out", drop.y_dtype, n * drop.features, dev)
    ly._call("tpconv_dropout_forward", dev, stream, drop.handle, n, x.data_ptr(), rng.data_ptr(), ly._ptr(residual),
             out.data_ptr())
    return out


def tpconv_dropout_backward(drop: Dropout, grad_y, rng, grad_x=None, stream=None):
    """The gradient of x, fp32, in grad_y's shape; rng as its forward had it.  grad_x may be grad_y."""
    dev = ly._device(grad_y, "grad_y")
    n = _dropout_nodes(drop, grad_y, "grad_y")
    ly._need(grad_y, "grad_y", torch.float32, n * drop.features, dev)
    ly._need(rng, "rng", torch.int64, 2, dev)
    if grad_x is None:
        grad_x = ly._new(grad_y.shape, torch.float32, dev, stream, grad_y)
    else:
        ly._need(grad_x, "grad_x", torch.float32, n * drop.features, dev)
    ly._call("tpconv_dropout_backward", dev, stream, drop.handle, n, grad_y.data_ptr(), rng.data_ptr(),
             grad_x.data_ptr())
    return grad_x
