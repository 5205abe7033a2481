"""Binding of the training-step operators (C ABI in ``include/ra_operators.h``):
the embedding and its gradient, the linear layer and its gradients on the
tensor cores, and activation checkpoints in 8 bits.

As in the rest of the package the functions carry the C names and only marshal
arguments.  Matrices are two-dimensional CUDA tensors, float32 or bfloat16 as
each call says, whose rows are contiguous (any row stride, so slices of a
larger tensor work); the outputs are allocated here unless ``out`` is given.
Work goes to the current torch stream unless ``stream`` is given; what is
allocated here is allocated for that stream, and a tensor that another stream
made or still uses needs the usual event or ``record_stream``.  The tensors
have to be on the current device: the library launches there.
"""
from __future__ import annotations

import ctypes

import torch

import gradient_ring_all_gb300 as _ra

ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "silu": 3}
GROUP = 32  # values of a row that share a checkpoint's step

_LARGE = 1 << 34  # for products below this ra_linear_split_bytes is not asked: a split would not repay the allocation

_F32, _BF16 = torch.float32, torch.bfloat16
_CODE = {_F32: 0, _BF16: 1}
_ID_BYTES = {torch.int32: 4, torch.int64: 8}
_CUDA = torch.device("cuda")  # the current device
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else None
_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device


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
    lib.ra_linear_split_bytes.argtypes = [i64, i64, i64]
    lib.ra_linear.argtypes = [vp, i64, vp, i64, i64, i64, i64, vp, i32, i32, vp, i64, i32, vp, vp, vp, i64, i32, vp, sz, vp]
    lib.ra_linear_dgrad.argtypes = [vp, i64, vp, i64, i64, i64, i64, vp, vp, i32, vp, i64, i32, vp, i64, i32, vp, sz, vp]
    lib.ra_linear_wgrad.argtypes = [vp, i64, vp, vp, i32, vp, i64, i64, i64, i64, i32, vp, i64, i32, vp, vp, sz, vp]
    lib.ra_selftest_linear_stall.argtypes = [i32, i32]
    for name in ("ra_checkpoint8_pack", "ra_checkpoint8_unpack", "ra_embedding_lookup", "ra_embedding_grad", "ra_linear",
                 "ra_linear_dgrad", "ra_linear_wgrad", "ra_selftest_linear_stall"):
        getattr(lib, name).restype = i32
    for name in ("ra_embedding_grad_workspace_bytes", "ra_linear_workspace_bytes", "ra_linear_split_bytes"):
        getattr(lib, name).restype = sz
    _declared = lib
    return lib


# ---------------------------------------------------------------------------
# marshalling (it runs on every call, and a small call takes the GPU less time
# than the host: one look at each attribute)


def _device(dev):
    """The number of the call's device (-1: the host, which the tensors' own checks refuse)."""
    if dev >= 0 and dev != _current_device():
        raise ValueError("the call's tensors are on cuda:%d, the current device is cuda:%d" % (dev, _current_device()))
    return dev


def _matrix(t, what, dev, dtype, shape):
    """(pointer, row stride, type code) of a matrix of the given shape on device number `dev`."""
    code = _CODE.get(t.dtype)
    if code is None or (dtype is not None and t.dtype != dtype):
        raise TypeError("%s must be %s, got %s" % (what, dtype or "float32 or bfloat16", t.dtype))
    if t.get_device() != dev or dev < 0:
        raise ValueError("%s must be a CUDA tensor on the call's device" % what)
    s = t.shape
    if s != shape:
        raise ValueError("%s must be a matrix of shape %s, got %s" % (what, tuple(shape), tuple(s)))
    ld, one = t.stride()
    if (one != 1 and s[1] > 1) or (ld < s[1] and s[0] > 1):
        raise ValueError("%s must have contiguous rows that do not overlap, got strides %s" % (what, (ld, one)))
    return t.data_ptr(), ld, code


def _shape(t, what):
    s = t.shape
    if len(s) != 2:
        raise ValueError("%s must be a matrix, got shape %s" % (what, tuple(s)))
    return s


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


def _output(out, rows, cols, dtype, like, dev, stream, what="out"):
    """(tensor, pointer, row stride, type code) of the output given, or of a new one beside `like`; `dtype`: the type wanted."""
    if out is None:
        code = _CODE.get(dtype)
        if code is None:
            raise TypeError("dtype must be float32 or bfloat16, got %s" % dtype)
        out = _empty((rows, cols), dtype, like.device, stream)
        return out, out.data_ptr(), cols, code
    return (out, *_matrix(out, what, dev, dtype, (rows, cols)))


def _act(act):
    code = ACTIVATIONS.get(act)
    if code is None:
        raise ValueError("act must be one of %s, got %r" % (", ".join(ACTIVATIONS), act))
    return code


def _ids(ids, dev):
    size = _ID_BYTES.get(ids.dtype)
    if size is None:
        raise TypeError("ids must be int32 or int64, got %s" % ids.dtype)
    if ids.get_device() != dev or dev < 0:
        raise ValueError("ids must be a CUDA tensor on the call's device")
    if not ids.is_contiguous():
        raise ValueError("ids must be contiguous")
    return ids.data_ptr(), size, ids.numel()


def _stream_of(stream, index):
    if stream is None:
        return _raw_stream(index) if _raw_stream else torch.cuda.current_stream(index).cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


def _in_place(p, ld, rows):
    """Whether TMA can read a bf16 matrix where it lies (rows on 16-byte boundaries)."""
    return p % 16 == 0 and (ld % 8 == 0 or rows <= 1)


def _workspace(workspace, need, like, stream):
    """(tensor to hold, pointer, bytes)."""
    if workspace is None:
        workspace = _empty((need,), torch.uint8, like.device, stream)
        return workspace, workspace.data_ptr(), need
    if not workspace.is_cuda or workspace.device != like.device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor on the call's device")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _room(workspace, in_place, rows, cols, k, mkn, like, stream, lib):
    """The linear layer's workspace: (tensor to hold, pointer, bytes), none where it helps nothing."""
    if workspace is None:
        need = 0 if in_place else lib.ra_linear_workspace_bytes(*mkn)
        if rows * cols * k >= _LARGE:
            need += lib.ra_linear_split_bytes(rows, cols, k)
        if need == 0:
            return None, None, 0
    else:
        need = 0
    return _workspace(workspace, need, like, stream)


def _check(status, what):
    if status:
        raise _ra.RaError(status, what)


# ---------------------------------------------------------------------------
# activation checkpoints


class Checkpoint8:
    """A rows x cols activation in 8 bits: ``q`` int8 [rows, groups * 32] and
    ``e`` uint8 [rows, groups], groups = ceil(cols / 32); group g of a row
    stands for q * 2**(e - 127).  New arrays are allocated (and not set) on
    `device` unless both are given."""

    __slots__ = ("rows", "cols", "_q", "_e", "_buffer", "_pq", "_pe", "_dev")

    def __init__(self, rows: int, cols: int, q=None, e=None, device=None):
        groups = -(-cols // GROUP)
        self.rows, self.cols, self._q, self._e = rows, cols, q, e
        if q is None and e is None:
            count = rows * groups
            self._buffer = b = torch.empty(count * (GROUP + 1), dtype=torch.uint8, device=_CUDA if device is None else device)
            self._pq = p = b.data_ptr()
            self._pe = p + count * GROUP
            self._dev = b.get_device()
            if self._dev < 0:
                raise ValueError("a checkpoint must be on a CUDA device")
            return
        if q is None or e is None:
            raise ValueError("give both q and e, or neither")
        if q.dtype != torch.int8 or q.shape != (rows, groups * GROUP) or not q.is_contiguous():
            raise ValueError("q must be a contiguous int8 tensor of shape %s" % ((rows, groups * GROUP),))
        if e.dtype != torch.uint8 or e.shape != (rows, groups) or not e.is_contiguous():
            raise ValueError("e must be a contiguous uint8 tensor of shape %s" % ((rows, groups),))
        self._dev = q.get_device()
        if self._dev < 0 or e.get_device() != self._dev:
            raise ValueError("q and e must be on one CUDA device")
        self._buffer, self._pq, self._pe = None, q.data_ptr(), e.data_ptr()

    @property
    def q(self):
        if self._q is None:
            groups = -(-self.cols // GROUP)
            self._q = self._buffer[:self.rows * groups * GROUP].view(torch.int8).view(self.rows, groups * GROUP)
        return self._q

    @property
    def e(self):
        if self._e is None:
            groups = -(-self.cols // GROUP)
            self._e = self._buffer[self.rows * groups * GROUP:].view(self.rows, groups)
        return self._e

    @property
    def device(self):
        return (self._q if self._buffer is None else self._buffer).device

    @property
    def shape(self):
        return (self.rows, self.cols)


def _kept(c, what, rows, cols, dev):
    if not isinstance(c, Checkpoint8):
        raise TypeError("%s must be a Checkpoint8" % what)
    if c.rows != rows or c.cols != cols or c._dev != dev:
        raise ValueError("%s must be a checkpoint of shape %s on the call's device, got %s" % (what, (rows, cols), c.shape))
    return c._pq, c._pe


def ra_checkpoint8_pack(x, out=None, stream=None) -> Checkpoint8:
    """The 8-bit form of the matrix x (float32 or bfloat16): values are off by
    at most half a step, 1/127.5 of a group's largest magnitude (three times
    that in a group that reaches 255 * 2**120; see the C header)."""
    rows, cols = s = _shape(x, "x")
    dev = _device(x.get_device())
    p, ld, code = _matrix(x, "x", dev, None, s)
    if out is None:
        if stream is None:
            out = Checkpoint8(rows, cols, device=x.device)
        else:
            with _on(stream, x.device):
                out = Checkpoint8(rows, cols, device=x.device)
        q, e = out._pq, out._pe
    else:
        q, e = _kept(out, "out", rows, cols, dev)
    _check(_load().ra_checkpoint8_pack(p, ld, code, rows, cols, q, e, _stream_of(stream, dev)), "ra_checkpoint8_pack")
    return out


def ra_checkpoint8_unpack(kept, act="none", dtype=None, out=None, stream=None):
    """act(the values a checkpoint stands for), as a matrix of `dtype`
    (bfloat16 unless given, exact without an activation)."""
    if not isinstance(kept, Checkpoint8):
        raise TypeError("kept must be a Checkpoint8")
    dev, rows, cols = _device(kept._dev), kept.rows, kept.cols
    out, p, ld, code = _output(out, rows, cols, dtype or (_BF16 if out is None else None), kept, dev, stream)
    _check(_load().ra_checkpoint8_unpack(kept._pq, kept._pe, rows, cols, _act(act), p, ld, code, _stream_of(stream, dev)),
           "ra_checkpoint8_unpack")
    return out


# ---------------------------------------------------------------------------
# embedding


def ra_embedding_lookup(table, ids, scale: float = 1.0, out=None, stream=None):
    """scale * table[ids]: one row per id (ids of any shape, flattened), zeros
    for an id outside the table (padding)."""
    vocab, d = s = _shape(table, "table")
    dev = _device(table.get_device())
    pt, ldt, code = _matrix(table, "table", dev, None, s)
    pi, size, count = _ids(ids, dev)
    out, po, ldo, _ = _output(out, count, d, table.dtype, table, dev, stream)
    _check(_load().ra_embedding_lookup(pt, ldt, code, vocab, d, pi, size, count, scale, po, ldo, _stream_of(stream, dev)),
           "ra_embedding_lookup")
    return out


def ra_embedding_grad(grad, ids, vocab: int, scale: float = 1.0, dtype=None, out=None, accumulate: bool = False, workspace=None,
                      stream=None):
    """The gradient of ra_embedding_lookup: row v is scale times the sum of
    grad's rows whose id is v, in token order; zero where there is none.
    `out` may be a view of a worker's flat gradient; accumulate adds to it.
    dtype: the new output's type (grad's unless given)."""
    rows, d = s = _shape(grad, "grad")
    dev = _device(grad.get_device())
    pg, ldg, gcode = _matrix(grad, "grad", dev, None, s)
    pi, size, count = _ids(ids, dev)
    if rows != count:
        raise ValueError("grad must have one row for each of the %d ids, got %d" % (count, rows))
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    out, po, ldo, ocode = _output(out, vocab, d, dtype or (grad.dtype if out is None else None), grad, dev, stream)
    lib = _load()
    hold, pw, nw = _workspace(workspace, lib.ra_embedding_grad_workspace_bytes(count, vocab, d), grad, stream)
    _check(lib.ra_embedding_grad(pg, ldg, gcode, pi, size, count, scale, int(accumulate), po, ldo, ocode, vocab, d, pw, nw,
                                 _stream_of(stream, dev)), "ra_embedding_grad")
    return out


# ---------------------------------------------------------------------------
# linear layer


def ra_linear(x, w, bias=None, act="none", residual=None, save=None, dtype=None, out=None, workspace=None, stream=None):
    """act(x @ w + bias) + residual, x [m, k] and w [k, n] bfloat16.  `save`, a
    Checkpoint8 of shape (m, n), receives x @ w + bias in 8 bits.  `out` may be
    the residual itself."""
    m, k = s = _shape(x, "x")
    dev = _device(x.get_device())
    px, ldx, _ = _matrix(x, "x", dev, _BF16, s)
    n = w.shape[-1]
    pw, ldw, _ = _matrix(w, "w", dev, _BF16, (k, n))
    pb, bcode, pr, ldr, rcode, pq, pe = None, 0, None, 0, 0, None, None
    if bias is not None:
        bcode = _CODE.get(bias.dtype)
        if bcode is None or bias.shape != (n,) or bias.get_device() != dev or not bias.is_contiguous():
            raise ValueError("bias must be a contiguous float32 or bfloat16 CUDA vector of length %d" % n)
        pb = bias.data_ptr()
    if residual is not None:
        pr, ldr, rcode = _matrix(residual, "residual", dev, None, (m, n))
    if save is not None:
        pq, pe = _kept(save, "save", m, n, dev)
    out, py, ldy, ycode = _output(out, m, n, dtype or (_BF16 if out is None else None), x, dev, stream)
    lib = _load()
    hold, ws, nws = _room(workspace, _in_place(px, ldx, m) and _in_place(pw, ldw, k), m, n, k, (m, k, n), x, stream, lib)
    _check(lib.ra_linear(px, ldx, pw, ldw, m, k, n, pb, bcode, _act(act), pr, ldr, rcode, pq, pe, py, ldy, ycode, ws, nws,
                         _stream_of(stream, dev)), "ra_linear")
    return out


def ra_linear_dgrad(dy, w, saved=None, act="none", residual=None, dtype=None, out=None, workspace=None, stream=None):
    """(dy @ w.T) * act'(z) + residual, dy [m, n] and w [k, n] bfloat16; z is
    the checkpoint `saved` of shape (m, k) (not needed with act "none")."""
    m, n = s = _shape(dy, "dy")
    dev = _device(dy.get_device())
    pd, ldd, _ = _matrix(dy, "dy", dev, _BF16, s)
    k = w.shape[0]
    pw, ldw, _ = _matrix(w, "w", dev, _BF16, (k, n))
    code = _act(act)
    pr, ldr, rcode, pq, pe = None, 0, 0, None, None
    if saved is not None:
        pq, pe = _kept(saved, "saved", m, k, dev)
    elif code:
        raise ValueError("act %r needs the checkpoint `saved`" % act)
    if residual is not None:
        pr, ldr, rcode = _matrix(residual, "residual", dev, None, (m, k))
    out, px, ldx, xcode = _output(out, m, k, dtype or (_BF16 if out is None else None), dy, dev, stream)
    lib = _load()
    hold, ws, nws = _room(workspace, _in_place(pd, ldd, m) and _in_place(pw, ldw, k), m, k, n, (m, k, n), dy, stream, lib)
    _check(lib.ra_linear_dgrad(pd, ldd, pw, ldw, m, k, n, pq, pe, code, pr, ldr, rcode, px, ldx, xcode, ws, nws,
                               _stream_of(stream, dev)), "ra_linear_dgrad")
    return out


def ra_linear_wgrad(x, dy, act="none", dtype=None, out=None, bias_grad=False, accumulate: bool = False, workspace=None, stream=None):
    """a.T @ dy, and with `bias_grad` also the column sums of dy: (dw, db).
    x is the layer's input [m, k] in bfloat16 (a = x) or the Checkpoint8 of z
    (a = act(z), rounded to bfloat16 also where dw is float32); dy [m, n]
    bfloat16.  `out` (dw) may be a view of a worker's flat gradient; bias_grad
    True or a float32 vector of length n that receives db; accumulate adds to
    both."""
    m, n = s = _shape(dy, "dy")
    dev = _device(dy.get_device())
    pd, ldd, _ = _matrix(dy, "dy", dev, _BF16, s)
    k = x.shape[1]
    code = _act(act)
    px, ldx, pq, pe = None, 0, None, None
    if isinstance(x, Checkpoint8):
        pq, pe = _kept(x, "x", m, k, dev)
    else:
        if code:
            raise ValueError("act %r needs x to be the Checkpoint8 of z" % act)
        px, ldx, _ = _matrix(x, "x", dev, _BF16, (m, k))
    if accumulate and (out is None or bias_grad is True):
        raise ValueError("accumulate needs out, and db's vector where db is wanted")
    out, pw, ldw, wcode = _output(out, k, n, dtype or (_BF16 if out is None else None), dy, dev, stream)
    pb, db = None, None
    if bias_grad is True:
        db = _empty((n,), _F32, dy.device, stream)
        pb = db.data_ptr()
    elif bias_grad is not False and bias_grad is not None:
        db = bias_grad
        if db.shape != (n,) or db.get_device() != dev or db.dtype != _F32 or not db.is_contiguous():
            raise ValueError("bias_grad must be True or a contiguous float32 CUDA vector of length %d" % n)
        pb = db.data_ptr()
    lib = _load()
    hold, ws, nws = _room(workspace, px is not None and _in_place(px, ldx, m) and _in_place(pd, ldd, m), k, n, m, (m, k, n), dy, stream, lib)
    _check(lib.ra_linear_wgrad(px, ldx, pq, pe, code, pd, ldd, m, k, n, int(accumulate), pw, ldw, wcode, pb, ws, nws,
                               _stream_of(stream, dev)), "ra_linear_wgrad")
    return out if pb is None else (out, db)


def ra_selftest_linear_stall(block: int, timeout_us: int) -> None:
    """Let this thread's next product run out of time: block `block` of its grid makes no copies, and its waits are limited to
    timeout_us (a timeout test)."""
    _check(_load().ra_selftest_linear_stall(int(block), int(timeout_us)), "ra_selftest_linear_stall")
