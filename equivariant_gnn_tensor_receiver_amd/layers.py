"""Python binding of the node layers (the C ABI in include/tpconv_layers.h): layer norm over irreps, a linear layer
with one weight matrix per group of nodes, and the orthogonalised (Muon) update of weight matrices.

As in ``tpconv``: argument marshalling only, functions carry the C names, PyTorch provides device memory and the
current HIP stream.  Tensors are contiguous; node tensors hold N * features values in any shape (results have the
features' shape of the layer, [N][F], or the shape of the input they belong to).
"""
from __future__ import annotations

import ctypes
from ctypes import POINTER, c_char_p, c_float, c_int32, c_int64, c_size_t, c_void_p

import torch

from . import tpconv as tp
from .tpconv import OP_BACKWARD, OP_FORWARD, TPCONV_BF16, TPCONV_F32  # noqa: F401  (part of this module's interface)

EXPORTS = ("tpconv_norm_create", "tpconv_norm_destroy", "tpconv_norm_info", "tpconv_norm_workspace_size",
           "tpconv_norm_forward", "tpconv_norm_backward", "tpconv_linear_create", "tpconv_linear_destroy",
           "tpconv_linear_info", "tpconv_linear_block", "tpconv_linear_groups_workspace_size",
           "tpconv_linear_groups", "tpconv_linear_workspace_size", "tpconv_linear_forward",
           "tpconv_linear_backward", "tpconv_muon_create", "tpconv_muon_destroy", "tpconv_muon_workspace_size",
           "tpconv_plan_weight_blocks", "tpconv_linear_weight_blocks", "tpconv_muon_orthogonalize",
           "tpconv_muon_step")

#: Quintic coefficients (a, b, c) of one step that drives singular values in (0, 1] towards 1, as published for the
#: Muon optimiser (K. Jordan et al., 2024); five steps are usual.
QUINTIC = (3.4445, -4.7750, 2.0315)


class NormDesc(ctypes.Structure):
    _fields_ = [("irreps", c_char_p), ("eps", c_float), ("x_dtype", c_int32), ("y_dtype", c_int32)]


class LinearDesc(ctypes.Structure):
    _fields_ = [("irreps_in", c_char_p), ("irreps_out", c_char_p), ("num_groups", c_int32), ("x_dtype", c_int32),
                ("w_dtype", c_int32), ("y_dtype", c_int32)]


class MatrixBlock(ctypes.Structure):
    _fields_ = [("rows", c_int32), ("cols", c_int32), ("count", c_int64), ("offset", c_int64), ("stride", c_int64)]


class MuonDesc(ctypes.Structure):
    _fields_ = [("num_blocks", c_int32), ("blocks", POINTER(MatrixBlock)), ("num_steps", c_int32),
                ("coefficients", POINTER(c_float)), ("eps", c_float)]


class MuonStepArgs(ctypes.Structure):
    _fields_ = [("lr", c_float), ("beta", c_float), ("nesterov", c_int32), ("weight_decay", c_float)]


_LIB = None


def _lib():
    global _LIB
    if _LIB is None:
        L = tp._lib()
        P, N, S = c_void_p, c_int64, c_size_t
        L.tpconv_norm_create.argtypes = [POINTER(P), POINTER(NormDesc)]
        L.tpconv_norm_destroy.argtypes = [P]
        L.tpconv_norm_info.argtypes = [P, POINTER(N), POINTER(c_int32), POINTER(N), POINTER(N)]
        L.tpconv_norm_workspace_size.argtypes = [P, N, POINTER(S)]
        L.tpconv_norm_forward.argtypes = [P, N, P, P, P, P, P, P]
        L.tpconv_norm_backward.argtypes = [P, N, P, P, P, P, P, P, P, P, S, P]
        L.tpconv_linear_create.argtypes = [POINTER(P), POINTER(LinearDesc)]
        L.tpconv_linear_destroy.argtypes = [P]
        L.tpconv_linear_info.argtypes = [P, POINTER(N), POINTER(N), POINTER(N), POINTER(c_int32)]
        L.tpconv_linear_block.argtypes = [P, c_int32, POINTER(c_int32), POINTER(c_int32), POINTER(N)]
        L.tpconv_linear_groups_workspace_size.argtypes = [P, N, POINTER(S)]
        L.tpconv_linear_groups.argtypes = [P, N, P, P, P, c_int32, P, S, P]
        L.tpconv_linear_workspace_size.argtypes = [P, c_int32, N, POINTER(S)]
        L.tpconv_linear_forward.argtypes = [P, N, P, P, P, P, P, P, S, P]
        L.tpconv_linear_backward.argtypes = [P, N, P, P, P, P, P, P, P, P, S, P]
        L.tpconv_muon_create.argtypes = [POINTER(P), POINTER(MuonDesc)]
        L.tpconv_muon_destroy.argtypes = [P]
        L.tpconv_muon_workspace_size.argtypes = [P, POINTER(S)]
        L.tpconv_plan_weight_blocks.argtypes = [P, POINTER(MatrixBlock), c_int32, POINTER(c_int32)]
        L.tpconv_linear_weight_blocks.argtypes = [P, POINTER(MatrixBlock), c_int32, POINTER(c_int32)]
        L.tpconv_muon_orthogonalize.argtypes = [P, P, P, P, S, P]
        L.tpconv_muon_step.argtypes = [P, POINTER(MuonStepArgs), P, P, P, P, P, P, P, S, P]
        for name in EXPORTS:
            getattr(L, name).restype = c_int32
        _LIB = L
    return _LIB


class _Handle:
    """Owning handle of a host-side object of the library (no device memory)."""

    handle = None
    _destroy = ""

    def __del__(self):
        if self.handle is not None and _LIB is not None:
            getattr(_LIB, self._destroy)(self.handle)
            self.handle = None


def _dtype(code):
    return torch.bfloat16 if code == TPCONV_BF16 else torch.float32


def _need(t, name, dtype, numel, device):
    # one test on the usual path; the shared check names what is wrong
    if t.dtype != dtype or t.numel() != numel or t.device != device or not t.is_contiguous():
        tp._require(t, name, dtype, numel, device)


def _device(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name}: on {t.device}, expected a GPU")
    return t.device


_raw_stream = torch._C._cuda_getCurrentRawStream  # the current stream's handle without a Stream object


def _call(fn, device, stream, *args):
    """fn(*args, stream) on the tensors' device, on `stream` or that device's current stream."""
    index = device.index
    handle = _raw_stream(index) if stream is None else stream.cuda_stream
    if torch.cuda.current_device() == index:
        st = getattr(_LIB, fn)(*args, handle)
    else:
        with torch.cuda.device(device):
            st = getattr(_LIB, fn)(*args, handle)
    if st != 0:
        raise tp.TpconvError(st, fn)


def _on(stream, device, make):
    """make(): a new tensor (and what fills it) for a call on `stream`.  Its memory comes from that stream's pool, since
    pending work of the current stream may still use what the current one's holds, and stays until the current stream,
    on which a result is used as well, is done with it."""
    if stream is None:
        return make()
    with torch.cuda.stream(stream):
        t = make()
    t.record_stream(torch.cuda.current_stream(device))
    return t


def _new(shape, dtype, device, stream, like=None):
    """An uninitialised result."""
    if stream is not None:
        return _on(stream, device, lambda: _new(shape, dtype, device, None, like))
    if like is not None and like.dtype == dtype:
        return torch.empty_like(like)
    return torch.empty(shape, dtype=dtype, device=device)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _nothing_to_compute(*outs):
    """Whether every wanted result is empty (an empty tensor has no address, which C reads as one that is not wanted)."""
    wanted = [t for t in outs if t is not None]
    return bool(wanted) and all(t.numel() == 0 for t in wanted)


def _scratch(workspace, need, device, stream):
    """(workspace, bytes): the caller's, or a new one of `need` bytes."""
    if workspace is None:
        if need == 0:
            return None, 0
        workspace = _new(need, torch.uint8, device, stream)
    elif workspace.device != device or not workspace.is_contiguous():
        tp._require(workspace, "workspace", None, None, device)
    return workspace, workspace.nbytes


# ---- layer norm ---------------------------------------------------------------------


class Norm(_Handle):
    """Layer norm over the irreps of a node tensor [N][F]."""

    _destroy = "tpconv_norm_destroy"

    def __init__(self, irreps: str, eps: float = 1e-5, x_dtype: int = TPCONV_F32, y_dtype: int = TPCONV_F32):
        L, h = _lib(), c_void_p()
        desc = NormDesc(irreps.encode(), eps, x_dtype, y_dtype)
        tp._check(L.tpconv_norm_create(ctypes.byref(h), ctypes.byref(desc)), "tpconv_norm_create")
        self.handle = h
        f, n, w, b = c_int64(), c_int32(), c_int64(), c_int64()
        tp._check(L.tpconv_norm_info(h, *(ctypes.byref(v) for v in (f, n, w, b))), "tpconv_norm_info")
        self.features, self.num_irreps, self.num_weights, self.num_biases = f.value, n.value, w.value, b.value
        self.x_dtype, self.y_dtype = _dtype(x_dtype), _dtype(y_dtype)
        self._ws = (None, 0)

    def stats_shape(self, num_nodes: int):
        """Shape of the statistics a forward can save: (mean, 1 / deviation) per node and irrep."""
        return (num_nodes, self.num_irreps, 2)

    def workspace_size(self, num_nodes: int) -> int:
        last, size = self._ws  # one read and one store: other threads may ask the same handle
        if last != num_nodes:
            b = c_size_t()
            tp._check(_LIB.tpconv_norm_workspace_size(self.handle, num_nodes, ctypes.byref(b)),
                      "tpconv_norm_workspace_size")
            size = b.value
            self._ws = (num_nodes, size)
        return size


def _norm_nodes(norm, x):
    n, rest = divmod(x.numel(), norm.features)
    if rest:
        raise ValueError(f"x: {x.numel()} elements, not a multiple of the {norm.features} features of a node")
    return n


def tpconv_norm_forward(norm: Norm, x, weight=None, bias=None, out=None, stats=None, stream=None):
    """norm(x), in x's shape.  stats: fp32 tensor of norm.stats_shape(N) that receives the statistics."""
    dev = _device(x, "x")
    n = _norm_nodes(norm, x)
    _need(x, "x", norm.x_dtype, n * norm.features, dev)
    if out is None:
        out = _new(x.shape, norm.y_dtype, dev, stream, x)
    else:
        _need(out, "out", norm.y_dtype, n * norm.features, dev)
    if weight is not None:
        _need(weight, "weight", torch.float32, norm.num_weights, dev)
    if bias is not None:
        _need(bias, "bias", torch.float32, norm.num_biases, dev)
    if stats is not None:
        _need(stats, "stats", torch.float32, 2 * n * norm.num_irreps, dev)
    _call("tpconv_norm_forward", dev, stream, norm.handle, n, x.data_ptr(), _ptr(weight), _ptr(bias),
          out.data_ptr(), _ptr(stats))
    return out


def tpconv_norm_backward(norm: Norm, x, weight, grad_y, stats=None, want=("x", "weight", "bias"), workspace=None,
                         stream=None, grad_x=None, grad_weight=None, grad_bias=None):
    """(grad_x, grad_weight, grad_bias) for the names in `want`, fp32; the others are None."""
    dev = _device(x, "x")
    n = _norm_nodes(norm, x)
    _need(x, "x", norm.x_dtype, n * norm.features, dev)
    _need(grad_y, "grad_y", torch.float32, n * norm.features, dev)
    if grad_x is None and "x" in want:
        grad_x = _new(x.shape, torch.float32, dev, stream, x)
    if grad_weight is None and "weight" in want:
        grad_weight = _new(norm.num_weights, torch.float32, dev, stream)
    if grad_bias is None and "bias" in want:
        grad_bias = _new(norm.num_biases, torch.float32, dev, stream)
    if weight is not None:
        _need(weight, "weight", torch.float32, norm.num_weights, dev)
    if stats is not None:
        _need(stats, "stats", torch.float32, 2 * n * norm.num_irreps, dev)
    if grad_x is not None:
        _need(grad_x, "grad_x", torch.float32, n * norm.features, dev)
    if grad_weight is not None:
        _need(grad_weight, "grad_weight", torch.float32, norm.num_weights, dev)
    if grad_bias is not None:
        _need(grad_bias, "grad_bias", torch.float32, norm.num_biases, dev)
    if _nothing_to_compute(grad_x, grad_weight, grad_bias):
        return grad_x, grad_weight, grad_bias
    need = norm.workspace_size(n) if grad_weight is not None or grad_bias is not None else 0
    workspace, nbytes = _scratch(workspace, need, dev, stream)
    _call("tpconv_norm_backward", dev, stream, norm.handle, n, x.data_ptr(), _ptr(weight), grad_y.data_ptr(),
          _ptr(stats), _ptr(grad_x), _ptr(grad_weight), _ptr(grad_bias), _ptr(workspace), nbytes)
    return grad_x, grad_weight, grad_bias


# ---- grouped linear layer -------------------------------------------------------------


class Linear(_Handle):
    """Linear layer between irreps with one weight matrix per (group, pair of irreps of equal degree and parity)."""

    _destroy = "tpconv_linear_destroy"

    def __init__(self, irreps_in: str, irreps_out: str, num_groups: int = 1, x_dtype: int = TPCONV_F32,
                 w_dtype: int = TPCONV_F32, y_dtype: int = TPCONV_F32):
        L, h = _lib(), c_void_p()
        desc = LinearDesc(irreps_in.encode(), irreps_out.encode(), num_groups, x_dtype, w_dtype, y_dtype)
        tp._check(L.tpconv_linear_create(ctypes.byref(h), ctypes.byref(desc)), "tpconv_linear_create")
        self.handle = h
        fi, fo, w, b = c_int64(), c_int64(), c_int64(), c_int32()
        tp._check(L.tpconv_linear_info(h, *(ctypes.byref(v) for v in (fi, fo, w, b))), "tpconv_linear_info")
        self.feat_in, self.feat_out, self.w_per_group, self.num_blocks = fi.value, fo.value, w.value, b.value
        self.num_groups = num_groups
        self.w_shape = (num_groups, self.w_per_group)
        self.x_dtype, self.w_dtype, self.y_dtype = _dtype(x_dtype), _dtype(w_dtype), _dtype(y_dtype)
        self._ws = {}

    def block(self, i: int):
        """((input irrep, output irrep), (mul_in, mul_out), offset within a group's weights) of weight block i."""
        idx, shape, off = (c_int32 * 2)(), (c_int32 * 2)(), c_int64()
        tp._check(_LIB.tpconv_linear_block(self.handle, i, idx, shape, ctypes.byref(off)), "tpconv_linear_block")
        return tuple(idx), tuple(shape), off.value

    def workspace_size(self, num_nodes: int, op: int = OP_BACKWARD) -> int:
        """Bytes for `op`; the backward's cover the forward too."""
        key = (num_nodes, op)
        size = self._ws.get(key)  # other threads may ask the same handle, and replace the dict
        if size is None:
            b = c_size_t()
            tp._check(_LIB.tpconv_linear_workspace_size(self.handle, op, num_nodes, ctypes.byref(b)),
                      "tpconv_linear_workspace_size")
            size = b.value
            if len(self._ws) > 16:
                self._ws = {}
            self._ws[key] = size
        return size


class Groups:
    """The nodes sorted by group (device int32): order [N], offsets [num_groups + 1]."""

    def __init__(self, num_nodes, offsets=None, order=None):
        self.num_nodes, self.offsets, self.order = num_nodes, offsets, order


def tpconv_linear_groups(linear: Linear, group, validate: bool = True, workspace=None, stream=None) -> Groups:
    """The grouping of the nodes with group ids `group` (int32 [N], 0..num_groups-1), for all later calls.  validate: ids
    outside the range raise (the call waits for the answer, so it cannot be captured); else such nodes are left out."""
    dev = _device(group, "group")
    n = group.numel()
    _need(group, "group", torch.int32, n, dev)
    offsets = _new(linear.num_groups + 1, torch.int32, dev, stream)
    order = _new(max(n, 1), torch.int32, dev, stream)
    b = c_size_t()
    tp._check(_LIB.tpconv_linear_groups_workspace_size(linear.handle, n, ctypes.byref(b)),
              "tpconv_linear_groups_workspace_size")
    workspace, nbytes = _scratch(workspace, b.value, dev, stream)
    _call("tpconv_linear_groups", dev, stream, linear.handle, n, group.data_ptr(), offsets.data_ptr(),
          order.data_ptr(), int(validate), _ptr(workspace), nbytes)
    return Groups(n, offsets, order)


def _linear_inputs(linear, groups, dev):
    n = groups.num_nodes
    if groups.offsets is not None:
        _need(groups.offsets, "offsets", torch.int32, linear.num_groups + 1, dev)
        _need(groups.order, "order", torch.int32, max(n, 1), dev)
    return n


def tpconv_linear_forward(linear: Linear, groups: Groups, x, W, out=None, workspace=None, stream=None):
    """y [N][F_out].  groups: of tpconv_linear_groups, or Groups(N) when there is one group."""
    dev = _device(x, "x")
    n = _linear_inputs(linear, groups, dev)
    _need(x, "x", linear.x_dtype, n * linear.feat_in, dev)
    _need(W, "W", linear.w_dtype, linear.num_groups * linear.w_per_group, dev)
    if out is None:
        out = _new((n, linear.feat_out), linear.y_dtype, dev, stream)
    else:
        _need(out, "out", linear.y_dtype, n * linear.feat_out, dev)
    workspace, nbytes = _scratch(workspace, linear.workspace_size(n, OP_FORWARD), dev, stream)
    _call("tpconv_linear_forward", dev, stream, linear.handle, n, _ptr(groups.offsets), _ptr(groups.order),
          x.data_ptr(), W.data_ptr(), out.data_ptr(), _ptr(workspace), nbytes)
    return out


def tpconv_linear_backward(linear: Linear, groups: Groups, x, W, grad_y, want=("x", "W"), workspace=None,
                           stream=None, grad_x=None, grad_W=None):
    """(grad_x in x's shape, grad_W [num_groups][w_per_group]) for the names in `want`, fp32; the others are None."""
    dev = _device(grad_y, "grad_y")
    n = _linear_inputs(linear, groups, dev)
    _need(grad_y, "grad_y", torch.float32, n * linear.feat_out, dev)
    _need(x, "x", linear.x_dtype, n * linear.feat_in, dev)
    _need(W, "W", linear.w_dtype, linear.num_groups * linear.w_per_group, dev)
    if grad_x is None and "x" in want:
        grad_x = _new(x.shape, torch.float32, dev, stream, x)
    if grad_W is None and "W" in want:
        grad_W = _new(linear.w_shape, torch.float32, dev, stream)
    if grad_x is not None:
        _need(grad_x, "grad_x", torch.float32, n * linear.feat_in, dev)
    if grad_W is not None:
        _need(grad_W, "grad_W", torch.float32, linear.num_groups * linear.w_per_group, dev)
    if _nothing_to_compute(grad_x, grad_W):
        return grad_x, grad_W
    workspace, nbytes = _scratch(workspace, linear.workspace_size(n) if grad_W is not None else 0, dev, stream)
    _call("tpconv_linear_backward", dev, stream, linear.handle, n, _ptr(groups.offsets), _ptr(groups.order),
          x.data_ptr(), W.data_ptr(), grad_y.data_ptr(), _ptr(grad_x), _ptr(grad_W), _ptr(workspace), nbytes)
    return grad_x, grad_W


# ---- orthogonalised update --------------------------------------------------------------


def weight_blocks(layer):
    """The weight matrices of a tpconv.Plan's W or a Linear's W, as Muon takes them."""
    if isinstance(layer, Linear):
        fn = _lib().tpconv_linear_weight_blocks
    else:
        fn = _lib().tpconv_plan_weight_blocks
    n = c_int32()
    tp._check(fn(layer.handle, None, 0, ctypes.byref(n)), "weight_blocks")
    b = (MatrixBlock * max(1, n.value))()
    tp._check(fn(layer.handle, b, n.value, ctypes.byref(n)), "weight_blocks")
    return [(v.rows, v.cols, v.count, v.offset, v.stride) for v in b[:n.value]]


class Muon(_Handle):
    """Orthogonalised momentum update of the matrices `blocks`: (rows, cols[, count[, offset[, stride]]]) each, in
    elements of the weight tensor (offset 0 and a stride of rows * cols when they are left out)."""

    _destroy = "tpconv_muon_destroy"

    def __init__(self, blocks, steps=(QUINTIC,) * 5, eps: float = 1e-7):
        L, h = _lib(), c_void_p()
        full = []
        for b in blocks:
            rows, cols, count, offset, stride = (*b, *(1, 0, b[0] * b[1])[len(b) - 2:])
            full.append(MatrixBlock(rows, cols, count, offset, stride))
        arr = (MatrixBlock * max(1, len(full)))(*full)
        steps = [tuple(s) for s in steps]
        if any(len(s) != 3 for s in steps):
            raise ValueError(f"steps: {steps}, expected (a, b, c) of every step")
        flat = [float(v) for s in steps for v in s]
        co = (c_float * max(1, len(flat)))(*flat)
        desc = MuonDesc(len(full), arr, len(steps), co, eps)
        tp._check(L.tpconv_muon_create(ctypes.byref(h), ctypes.byref(desc)), "tpconv_muon_create")
        self.handle = h
        #: elements a weight tensor must have at least
        self.numel = max((b.offset + (b.count - 1) * b.stride + b.rows * b.cols for b in full if b.count), default=0)
        #: elements the blocks cover: a tensor of exactly so many has none outside them
        self.dense = sum(b.count * b.rows * b.cols for b in full)
        n = c_size_t()
        tp._check(L.tpconv_muon_workspace_size(h, ctypes.byref(n)), "tpconv_muon_workspace_size")
        self._ws = n.value

    def workspace_size(self) -> int:
        return self._ws


def _muon_tensor(muon, t, name, dtype, numel, device):
    if numel < muon.numel:
        raise ValueError(f"{name}: {numel} elements, at least {muon.numel} needed")
    _need(t, name, dtype, numel, device)


def tpconv_muon_orthogonalize(muon: Muon, u, out=None, workspace=None, stream=None):
    """The matrices of u (fp32) orthogonalised, in u's shape; elements outside the blocks are zero in a new `out`."""
    dev = _device(u, "u")
    n = u.numel()
    _muon_tensor(muon, u, "u", torch.float32, n, dev)
    if out is None:
        if n == muon.dense:
            out = _new(u.shape, torch.float32, dev, stream, u)
        else:
            out = _on(stream, dev, lambda: torch.zeros_like(u))
    else:
        _muon_tensor(muon, out, "out", torch.float32, n, dev)
    if _nothing_to_compute(out):
        return out
    workspace, nbytes = _scratch(workspace, muon.workspace_size(), dev, stream)
    _call("tpconv_muon_orthogonalize", dev, stream, muon.handle, u.data_ptr(), out.data_ptr(), _ptr(workspace), nbytes)
    return out


def tpconv_muon_step(muon: Muon, W, grad, momentum, lr: float, beta: float = 0.95, nesterov: bool = True,
                     weight_decay: float = 0.0, W_out=None, momentum_out=None, W_bf16=None, workspace=None,
                     stream=None):
    """(new W, new momentum): new tensors, or W_out / momentum_out, which may be W / momentum themselves.  W_bf16
    receives the new weights in bf16 as well.  Elements outside the blocks keep their values in new tensors."""
    dev = _device(W, "W")
    n = W.numel()
    _muon_tensor(muon, W, "W", torch.float32, n, dev)
    _muon_tensor(muon, grad, "grad", torch.float32, n, dev)
    _muon_tensor(muon, momentum, "momentum", torch.float32, n, dev)
    dense = n == muon.dense
    if W_out is None:
        W_out = _new(W.shape, torch.float32, dev, stream, W) if dense else _on(stream, dev, W.clone)
    else:
        _muon_tensor(muon, W_out, "W_out", torch.float32, n, dev)
    if momentum_out is None:
        momentum_out = _new(W.shape, torch.float32, dev, stream, momentum) if dense else _on(stream, dev, momentum.clone)
    else:
        _muon_tensor(muon, momentum_out, "momentum_out", torch.float32, n, dev)
    if W_bf16 is not None:
        _muon_tensor(muon, W_bf16, "W_bf16", torch.bfloat16, n, dev)
    if _nothing_to_compute(W_out, momentum_out):
        return W_out, momentum_out
    workspace, nbytes = _scratch(workspace, muon.workspace_size(), dev, stream)
    args = MuonStepArgs(lr, beta, int(nesterov), weight_decay)
    _call("tpconv_muon_step", dev, stream, muon.handle, ctypes.byref(args), W.data_ptr(), grad.data_ptr(),
          momentum.data_ptr(), W_out.data_ptr(), momentum_out.data_ptr(), _ptr(W_bf16), _ptr(workspace), nbytes)
    return W_out, momentum_out
