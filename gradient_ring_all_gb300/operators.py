"""Binding of the training-step operators (C ABI in ``include/ra_operators.h``):
the embedding and its gradient, the linear layer and its gradients on the
tensor cores, and activation checkpoints in 8 bits.

As in the rest of the package the functions carry the C names and only marshal
arguments.  Matrices are two-dimensional CUDA tensors, float32 or bfloat16 as
each call says, whose rows are contiguous (any row stride, so slices of a
larger tensor work); the outputs are allocated here unless ``out`` is given.
Work goes to the current torch stream unless ``stream`` is given; what is
allocated here is allocated for that stream, and a tensor that another stream
made or still uses needs the usual event or ``record_stream``.
"""
from __future__ import annotations

import ctypes

import torch

import gradient_ring_all_gb300 as _ra

ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "silu": 3}
GROUP = 32  # values of a row that share a checkpoint's step

_F32, _BF16 = torch.float32, torch.bfloat16
_CODE = {_F32: 0, _BF16: 1}


_declared = None


def _load():
    """The loaded library, with the operators' C signatures set."""
    global _declared
    lib = _ra.load()
    if lib is _declared:
        return lib
    vp, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
    lib.ra_checkpoint8_pack.argtypes = [vp, i64, i32, i64, i64, vp, vp, vp]
    lib.ra_checkpoint8_unpack.argtypes = [vp, vp, i64, i64, i32, vp, i64, i32, vp]
    lib.ra_embedding_lookup.argtypes = [vp, i64, i32, i64, i64, vp, i32, i64, f32, vp, i64, vp]
    lib.ra_embedding_grad_workspace_bytes.argtypes = [i64, i64, i64]
    lib.ra_embedding_grad.argtypes = [vp, i64, i32, vp, i32, i64, f32, i32, vp, i64, i32, i64, i64, vp, sz, vp]
    lib.ra_linear_workspace_bytes.argtypes = [i64, i64, i64]
    lib.ra_linear.argtypes = [vp, i64, vp, i64, i64, i64, i64, vp, i32, i32, vp, i64, i32, vp, vp, vp, i64, i32, vp, sz, vp]
    lib.ra_linear_dgrad.argtypes = [vp, i64, vp, i64, i64, i64, i64, vp, vp, i32, vp, i64, i32, vp, i64, i32, vp, sz, vp]
    lib.ra_linear_wgrad.argtypes = [vp, i64, vp, vp, i32, vp, i64, i64, i64, i64, i32, vp, i64, i32, vp, vp, sz, vp]
    for name in ("ra_checkpoint8_pack", "ra_checkpoint8_unpack", "ra_embedding_lookup", "ra_embedding_grad", "ra_linear",
                 "ra_linear_dgrad", "ra_linear_wgrad"):
        getattr(lib, name).restype = i32
    for name in ("ra_embedding_grad_workspace_bytes", "ra_linear_workspace_bytes"):
        getattr(lib, name).restype = sz
    _declared = lib
    return lib


# ---------------------------------------------------------------------------
# marshalling


def _matrix(t, what, dev=None, dtype=None, shape=None):
    """(pointer, row stride, type code) of a matrix; checks what is asked of it."""
    if not t.is_cuda or (dev is not None and t.get_device() != dev):
        raise ValueError("%s must be a CUDA tensor on the call's device" % what)
    code = _CODE.get(t.dtype)
    if code is None or (dtype is not None and t.dtype != dtype):
        raise TypeError("%s must be %s, got %s" % (what, dtype or "float32 or bfloat16", t.dtype))
    if t.dim() != 2 or (shape is not None and tuple(t.shape) != shape):
        raise ValueError("%s must be a matrix%s, got shape %s" % (what, "" if shape is None else " of shape %s" % (shape,), tuple(t.shape)))
    ld, one = t.stride()
    if one != 1 and t.shape[1] > 1:
        raise ValueError("%s must have contiguous rows, got strides %s" % (what, t.stride()))
    if t.shape[0] > 1 and ld < t.shape[1]:
        raise ValueError("%s must have rows that do not overlap, got strides %s" % (what, t.stride()))
    return t.data_ptr(), ld, code


def _on(stream, dev):
    """The context in which a tensor for work on `stream` is allocated: torch's allocator then gives memory that this
    stream may use at once, and takes it back in this stream's order."""
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=dev) if stream else torch.cuda.default_stream(dev)
    return torch.cuda.stream(stream)


def _empty(shape, dtype, dev, stream):
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with _on(stream, dev):
        return torch.empty(shape, dtype=dtype, device=dev)


def _output(out, rows, cols, dtype, dev, what, stream):
    """The output given, or a new one; `dtype` is the type wanted, if any."""
    if out is None:
        return _empty((rows, cols), dtype or _BF16, dev, stream)
    if dtype is not None and out.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (what, dtype, out.dtype))
    return out


def _act(act):
    code = ACTIVATIONS.get(act)
    if code is None:
        raise ValueError("act must be one of %s, got %r" % (", ".join(ACTIVATIONS), act))
    return code


def _ids(ids, dev):
    if not ids.is_cuda or ids.get_device() != dev:
        raise ValueError("ids must be a CUDA tensor on the call's device")
    if ids.dtype == torch.int64:
        size = 8
    elif ids.dtype == torch.int32:
        size = 4
    else:
        raise TypeError("ids must be int32 or int64, got %s" % ids.dtype)
    if not ids.is_contiguous():
        raise ValueError("ids must be contiguous")
    return ids.data_ptr(), size, ids.numel()


def _stream_of(stream, index):
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(index)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _in_place(t):
    """Whether TMA can read a matrix where it lies (rows on 16-byte boundaries)."""
    return t.data_ptr() % 16 == 0 and (t.shape[0] <= 1 or t.stride(0) % 8 == 0)


def _workspace(workspace, need, dev, stream):
    """(tensor to hold, pointer, bytes)."""
    if workspace is None:
        workspace = _empty((need,), torch.uint8, dev, stream)
    elif not workspace.is_cuda or workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor on the call's device")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


# ---------------------------------------------------------------------------
# activation checkpoints


class Checkpoint8:
    """A rows x cols activation in 8 bits: ``q`` int8 [rows, groups * 32] and
    ``e`` uint8 [rows, groups], groups = ceil(cols / 32); group g of a row
    stands for q * 2**(e - 127).  New arrays are allocated (and not set)
    unless both are given."""

    __slots__ = ("rows", "cols", "q", "e")

    def __init__(self, rows: int, cols: int, q=None, e=None, device=None):
        groups = -(-cols // GROUP)
        if (q is None) != (e is None):
            raise ValueError("give both q and e, or neither")
        if q is None:
            device = torch.device("cuda", torch.cuda.current_device()) if device is None else device
            q = torch.empty(rows, groups * GROUP, dtype=torch.int8, device=device)
            e = torch.empty(rows, groups, dtype=torch.uint8, device=device)
        if q.dtype != torch.int8 or tuple(q.shape) != (rows, groups * GROUP) or not q.is_contiguous():
            raise ValueError("q must be a contiguous int8 tensor of shape %s" % ((rows, groups * GROUP),))
        if e.dtype != torch.uint8 or tuple(e.shape) != (rows, groups) or not e.is_contiguous() or e.device != q.device:
            raise ValueError("e must be a contiguous uint8 tensor of shape %s beside q" % ((rows, groups),))
        if not q.is_cuda:
            raise ValueError("a checkpoint must be on a CUDA device")
        self.rows, self.cols, self.q, self.e = rows, cols, q, e

    @property
    def device(self):
        return self.q.device

    @property
    def shape(self):
        return (self.rows, self.cols)


def _kept(c, what, shape, dev):
    if not isinstance(c, Checkpoint8):
        raise TypeError("%s must be a Checkpoint8" % what)
    if (c.rows, c.cols) != shape or c.q.get_device() != dev:
        raise ValueError("%s must be a checkpoint of shape %s on the call's device, got %s" % (what, shape, c.shape))
    return c.q.data_ptr(), c.e.data_ptr()


def ra_checkpoint8_pack(x, out=None, stream=None) -> Checkpoint8:
    """The 8-bit form of the matrix x (float32 or bfloat16): at most half a
    step, 1/127.5 of a group's largest magnitude, off."""
    p, ld, code = _matrix(x, "x")
    rows, cols = x.shape
    dev = x.get_device()
    if out is None:
        if stream is None:
            out = Checkpoint8(rows, cols, device=x.device)
        else:
            with _on(stream, x.device):
                out = Checkpoint8(rows, cols, device=x.device)
    q, e = _kept(out, "out", (rows, cols), dev)
    _ra._check(_load().ra_checkpoint8_pack(p, ld, code, rows, cols, q, e, _stream_of(stream, dev)), "ra_checkpoint8_pack")
    return out


def ra_checkpoint8_unpack(kept, act="none", dtype=None, out=None, stream=None):
    """act(the values a checkpoint stands for), as a matrix of `dtype`
    (bfloat16 unless given, exact without an activation)."""
    if not isinstance(kept, Checkpoint8):
        raise TypeError("kept must be a Checkpoint8")
    dev = kept.q.get_device()
    out = _output(out, kept.rows, kept.cols, dtype, kept.q.device, "out", stream)
    p, ld, code = _matrix(out, "out", dev, None, (kept.rows, kept.cols))
    _ra._check(_load().ra_checkpoint8_unpack(kept.q.data_ptr(), kept.e.data_ptr(), kept.rows, kept.cols, _act(act), p, ld, code,
                                                _stream_of(stream, dev)), "ra_checkpoint8_unpack")
    return out


# ---------------------------------------------------------------------------
# embedding


def ra_embedding_lookup(table, ids, scale: float = 1.0, out=None, stream=None):
    """scale * table[ids]: one row per id (ids of any shape, flattened), zeros
    for an id outside the table (padding)."""
    pt, ldt, code = _matrix(table, "table")
    dev = table.get_device()
    pi, size, count = _ids(ids, dev)
    vocab, d = table.shape
    out = _output(out, count, d, table.dtype, table.device, "out", stream)
    po, ldo, _ = _matrix(out, "out", dev, table.dtype, (count, d))
    _ra._check(_load().ra_embedding_lookup(pt, ldt, code, vocab, d, pi, size, count, scale, po, ldo, _stream_of(stream, dev)),
               "ra_embedding_lookup")
    return out


def ra_embedding_grad(grad, ids, vocab: int, scale: float = 1.0, dtype=None, out=None, accumulate: bool = False, workspace=None,
                      stream=None):
    """The gradient of ra_embedding_lookup: row v is scale times the sum of
    grad's rows whose id is v, in token order; zero where there is none.
    `out` may be a view of a worker's flat gradient; accumulate adds to it.
    dtype: the new output's type (grad's unless given)."""
    pg, ldg, gcode = _matrix(grad, "grad")
    dev = grad.get_device()
    pi, size, count = _ids(ids, dev)
    if grad.shape[0] != count:
        raise ValueError("grad must have one row for each of the %d ids, got %d" % (count, grad.shape[0]))
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    d = grad.shape[1]
    out = _output(out, vocab, d, dtype or (grad.dtype if out is None else None), grad.device, "out", stream)
    po, ldo, ocode = _matrix(out, "out", dev, None, (vocab, d))
    lib = _load()
    hold, pw, nw = _workspace(workspace, lib.ra_embedding_grad_workspace_bytes(count, vocab, d), grad.device, stream)
    _ra._check(lib.ra_embedding_grad(pg, ldg, gcode, pi, size, count, scale, int(accumulate), po, ldo, ocode, vocab, d, pw, nw,
                                     _stream_of(stream, dev)), "ra_embedding_grad")
    return out


# ---------------------------------------------------------------------------
# linear layer


def ra_linear(x, w, bias=None, act="none", residual=None, save=None, dtype=None, out=None, workspace=None, stream=None):
    """act(x @ w + bias) + residual, x [m, k] and w [k, n] bfloat16.  `save`, a
    Checkpoint8 of shape (m, n), receives x @ w + bias in 8 bits.  `out` may be
    the residual itself."""
    px, ldx, _ = _matrix(x, "x", None, _BF16)
    dev = x.get_device()
    m, k = x.shape
    n = w.shape[-1]
    pw, ldw, _ = _matrix(w, "w", dev, _BF16, (k, n))
    pb, bcode, pr, ldr, rcode, pq, pe = None, 0, None, 0, 0, None, None
    if bias is not None:
        if bias.dim() != 1 or bias.shape[0] != n or bias.get_device() != dev or not bias.is_contiguous() or bias.dtype not in _CODE:
            raise ValueError("bias must be a contiguous float32 or bfloat16 CUDA vector of length %d" % n)
        pb, bcode = bias.data_ptr(), _CODE[bias.dtype]
    if residual is not None:
        pr, ldr, rcode = _matrix(residual, "residual", dev, None, (m, n))
    if save is not None:
        pq, pe = _kept(save, "save", (m, n), dev)
    out = _output(out, m, n, dtype, x.device, "out", stream)
    py, ldy, ycode = _matrix(out, "out", dev, None, (m, n))
    lib = _load()
    ws, nws, hold = None, 0, None
    if workspace is not None or not (_in_place(x) and _in_place(w)):
        hold, ws, nws = _workspace(workspace, lib.ra_linear_workspace_bytes(m, k, n), x.device, stream)
    _ra._check(lib.ra_linear(px, ldx, pw, ldw, m, k, n, pb, bcode, _act(act), pr, ldr, rcode, pq, pe, py, ldy, ycode, ws, nws,
                             _stream_of(stream, dev)), "ra_linear")
    return out


def ra_linear_dgrad(dy, w, saved=None, act="none", residual=None, dtype=None, out=None, workspace=None, stream=None):
    """(dy @ w.T) * act'(z) + residual, dy [m, n] and w [k, n] bfloat16; z is
    the checkpoint `saved` of shape (m, k) (not needed with act "none")."""
    pd, ldd, _ = _matrix(dy, "dy", None, _BF16)
    dev = dy.get_device()
    m, n = dy.shape
    k = w.shape[0]
    pw, ldw, _ = _matrix(w, "w", dev, _BF16, (k, n))
    code = _act(act)
    pr, ldr, rcode, pq, pe = None, 0, 0, None, None
    if saved is not None:
        pq, pe = _kept(saved, "saved", (m, k), dev)
    elif code:
        raise ValueError("act %r needs the checkpoint `saved`" % act)
    if residual is not None:
        pr, ldr, rcode = _matrix(residual, "residual", dev, None, (m, k))
    out = _output(out, m, k, dtype, dy.device, "out", stream)
    px, ldx, xcode = _matrix(out, "out", dev, None, (m, k))
    lib = _load()
    ws, nws, hold = None, 0, None
    if workspace is not None or not (_in_place(dy) and _in_place(w)):
        hold, ws, nws = _workspace(workspace, lib.ra_linear_workspace_bytes(m, k, n), dy.device, stream)
    _ra._check(lib.ra_linear_dgrad(pd, ldd, pw, ldw, m, k, n, pq, pe, code, pr, ldr, rcode, px, ldx, xcode, ws, nws,
                                   _stream_of(stream, dev)), "ra_linear_dgrad")
    return out


def ra_linear_wgrad(x, dy, act="none", dtype=None, out=None, bias_grad=False, accumulate: bool = False, workspace=None, stream=None):
    """a.T @ dy, and with `bias_grad` also the column sums of dy: (dw, db).
    x is the layer's input [m, k] in bfloat16 (a = x) or the Checkpoint8 of z
    (a = act(z)); dy [m, n] bfloat16.  `out` (dw) may be a view of a worker's
    flat gradient; bias_grad True or a float32 vector of length n that receives
    db; accumulate adds to both."""
    pd, ldd, _ = _matrix(dy, "dy", None, _BF16)
    dev = dy.get_device()
    m, n = dy.shape
    k = x.shape[1]
    code = _act(act)
    px, ldx, pq, pe = None, 0, None, None
    if isinstance(x, Checkpoint8):
        pq, pe = _kept(x, "x", (m, k), dev)
    else:
        if code:
            raise ValueError("act %r needs x to be the Checkpoint8 of z" % act)
        px, ldx, _ = _matrix(x, "x", dev, _BF16, (m, k))
    if accumulate and (out is None or bias_grad is True):
        raise ValueError("accumulate needs out, and db's vector where db is wanted")
    out = _output(out, k, n, dtype, dy.device, "out", stream)
    pw, ldw, wcode = _matrix(out, "out", dev, None, (k, n))
    pb, db = None, None
    if bias_grad is not False and bias_grad is not None:
        db = _empty((n,), _F32, dy.device, stream) if bias_grad is True else bias_grad
        if db.dim() != 1 or db.shape[0] != n or db.get_device() != dev or db.dtype != _F32 or not db.is_contiguous():
            raise ValueError("bias_grad must be True or a contiguous float32 CUDA vector of length %d" % n)
        pb = db.data_ptr()
    lib = _load()
    ws, nws, hold = None, 0, None
    if workspace is not None or px is None or not (_in_place(x) and _in_place(dy)):
        hold, ws, nws = _workspace(workspace, lib.ra_linear_workspace_bytes(m, k, n), dy.device, stream)
    _ra._check(lib.ra_linear_wgrad(px, ldx, pq, pe, code, pd, ldd, m, k, n, int(accumulate), pw, ldw, wcode, pb, ws, nws,
                                   _stream_of(stream, dev)), "ra_linear_wgrad")
    return out if pb is None else (out, db)
