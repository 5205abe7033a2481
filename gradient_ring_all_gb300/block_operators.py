"""Binding of the operators between a training step's products (C ABI in
``include/ra_operators.h``): dropout, the norms around a block with its gate and
residual scale, and the log probabilities of given tokens, each with its
gradient.

The conventions are those of ``operators.py``.  A float's vector (a gain, a
row's log probability) is a contiguous one-dimensional CUDA tensor.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import operators as _op
from .operators import _BF16, _CODE, _F32, _check, _device, _empty, _ids, _matrix, _output, _shape, _stream_of, _workspace

KINDS = {"layer": 1, "rms": 2}
_KIND_NAMES = {code: kind for kind, code in KINDS.items()}
MAX_TOP = 32  # alternatives of a row

_NORM = "QQiifi"  # ra_norm
_BLOCK = struct.Struct("=qq" + "Qq" * 5 + "Q" + 2 * _NORM + "iiiiff")
_BLOCK_GRAD = struct.Struct("=qq" + "Qq" * 5 + "Q" + "Qq" * 3 + "QQQQQQ" + 2 * _NORM + "iiiiffii")
_NO_NORM = (0, 0, 0, 0, 0.0, 0)
_ROWS = torch.contiguous_format
# torch's allocator without a tensor around the memory (0.6 us instead of 2.7 a workspace)
_raw_alloc = getattr(torch._C, "_cuda_cudaCachingAllocator_raw_alloc", None)
_raw_delete = getattr(torch._C, "_cuda_cudaCachingAllocator_raw_delete", None)

_declared = None


def _load():
    """The loaded library, with these operators' C signatures set."""
    global _declared
    lib = _op._load()
    if lib is _declared:
        return lib
    vp, i32, i64, f32, f64, u32, u64 = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_double, ctypes.c_uint32,
                                        ctypes.c_uint64)
    lib.ra_dropout.argtypes = [vp, i64, i32, i64, i64, f64, u64, vp, u32, i64, vp, i64, i32, vp, i64, i32, vp]
    lib.ra_norm_block.argtypes = [ctypes.c_char_p, vp]
    lib.ra_norm_block_grad_workspace_bytes.argtypes = [i64, i64]
    lib.ra_norm_block_grad.argtypes = [ctypes.c_char_p, vp]
    lib.ra_logprobs.argtypes = [vp, i64, i32, i64, i64, vp, i32, f32, vp, vp, vp, i32, vp, vp, vp]
    lib.ra_logprobs_grad.argtypes = [vp, i64, i32, i64, i64, vp, i32, f32, vp, vp, vp, vp, vp, i64, i32, vp]
    for name in ("ra_dropout", "ra_norm_block", "ra_norm_block_grad", "ra_logprobs", "ra_logprobs_grad"):
        getattr(lib, name).restype = i32
    lib.ra_norm_block_grad_workspace_bytes.restype = ctypes.c_size_t
    _declared = lib
    return lib


def _vector(t, what, dev, n, dtype=None):
    """(pointer, type code) of a contiguous vector of n values."""
    code = _CODE.get(t.dtype)
    if code is None or (dtype is not None and t.dtype != dtype):
        raise TypeError("%s must be %s, got %s" % (what, dtype or "float32 or bfloat16", t.dtype))
    if t.get_device() != dev or dev < 0:
        raise ValueError("%s must be a CUDA tensor on the call's device" % what)
    if t.shape != (n,) or not t.is_contiguous():
        raise ValueError("%s must be a contiguous vector of length %d, got shape %s" % (what, n, tuple(t.shape)))
    return t.data_ptr(), code


def _like(t, what, dev, dtype, s):
    """(pointer, row stride) of a matrix of this type and shape: one look at what is right as a rule, _matrix says what is wrong."""
    if t.dtype is dtype and t.shape == s and t.get_device() == dev >= 0:
        ld, one = t.stride()
        if one == 1 and ld >= s[1]:
            return t.data_ptr(), ld
    return _matrix(t, what, dev, dtype, s)[:2]


# ---------------------------------------------------------------------------
# dropout


def ra_dropout(x, p: float, seed, site: int = 0, first_row: int = 0, residual=None, dtype=None, out=None, stream=None):
    """residual + x * keep / (1 - p), where the mask follows from the seed, the
    site and each value's row and column alone (the C header says how): the same
    call on the gradient, without the residual, is the backward pass.

    seed: a whole number of 64 bits, or a CUDA tensor with one int64, which is
    read when the kernel runs (a captured call then takes another mask at each
    replay).  first_row: the row of the mask that x's first row takes (a
    micro-batch's place in its batch).  p is rounded to a 65536th.  `out` may be
    x or the residual itself."""
    rows, cols = s = _shape(x, "x")
    dev = _device(x.get_device())
    px, ldx, xcode = _matrix(x, "x", dev, None, s)
    if not 0.0 <= p <= 1.0:
        raise ValueError("p must lie between 0 and 1, got %r" % (p,))
    if not 0 <= site < 1 << 32:
        raise ValueError("site must be a whole number of 32 bits, got %r" % (site,))
    if not 0 <= first_row < (1 << 63) - (1 << 31):
        raise ValueError("first_row must be at least 0 and below 2^63 - 2^31, got %r" % (first_row,))
    at = None
    if isinstance(seed, torch.Tensor):
        if seed.dtype != torch.int64 or seed.numel() != 1:
            raise TypeError("seed must be a whole number or an int64 tensor with one value, got %s of shape %s" % (seed.dtype, tuple(seed.shape)))
        if seed.get_device() != dev:
            raise ValueError("seed must be a CUDA tensor on the call's device")
        at, seed = seed.data_ptr(), 0
    elif not 0 <= seed < 1 << 64:
        raise ValueError("seed must be a whole number of 64 bits, got %r" % (seed,))
    pr, ldr, rcode = None, 0, 0
    if residual is not None:
        pr, ldr, rcode = _matrix(residual, "residual", dev, None, s)
    out, py, ldy, ycode = _output(out, rows, cols, dtype or (x.dtype if out is None else None), x, dev, stream)
    _check(_load().ra_dropout(px, ldx, xcode, rows, cols, p, seed, at, site, first_row, pr, ldr, rcode, py, ldy, ycode, _stream_of(stream, dev)),
           "ra_dropout")
    return out


# ---------------------------------------------------------------------------
# norms around a block


class Norm:
    """A norm over rows of d values: (v - m) * rstd * gain + bias, m the row's
    mean ("layer") or 0 ("rms"), rstd = (mean (v - m)^2 + eps)^-1/2.  gain and
    bias: vectors of one type (float32 or bfloat16), or None."""

    __slots__ = ("gain", "bias", "eps", "_kind")

    def __init__(self, gain=None, bias=None, kind: str = "layer", eps: float = 1e-5):
        if not 0.0 <= eps < float("inf"):
            raise ValueError("eps must be finite and not negative, got %r" % (eps,))
        self.gain, self.bias, self.eps, self._kind = gain, bias, eps, KINDS.get(kind) or self._unknown(kind)

    @staticmethod
    def _unknown(kind):
        raise ValueError("kind must be one of %s, got %r" % (", ".join(KINDS), kind))

    @property
    def kind(self):
        return _KIND_NAMES[self._kind]

    @kind.setter
    def kind(self, kind):
        self._kind = KINDS.get(kind) or self._unknown(kind)


def _norm(n, what, dev, d):
    """The fields of a ra_norm."""
    if n is None:
        return _NO_NORM
    if n.__class__ is not Norm and not isinstance(n, Norm):
        raise TypeError("%s must be a Norm" % what)
    gain, bias = n.gain, n.bias
    if gain is None:
        if bias is None:
            return 0, 0, 0, n._kind, n.eps, 0
        pb, code = _vector(bias, what + ".bias", dev, d)
        return 0, pb, code, n._kind, n.eps, 0
    pg, code = _vector(gain, what + ".gain", dev, d)
    return pg, 0 if bias is None else _vector(bias, what + ".bias", dev, d, gain.dtype)[0], code, n._kind, n.eps, 0


def _gate(gate, dev, rows, d, f):
    """(pointer, row stride, gate kind, type code)"""
    if gate is None:
        return 0, 0, 0, 0
    if gate.dim() == 1:
        p, code = _vector(gate, "gate", dev, d)
        return p, d, 1, code
    p, ld, code = _matrix(gate, "gate", dev, f.dtype, (rows, d))
    return p, ld, 2, code


def _new(like, dtype, stream):
    """A new matrix beside `like`, of its shape."""
    if stream is None and like.dtype is dtype:  # the quickest of torch's ways
        return torch.empty_like(like, memory_format=_ROWS)
    return _empty(like.shape, dtype, like.device, stream)


def _block_type(f, x):
    """The type of f and h beside a stream x."""
    if _CODE.get(f) is None or (f == _F32 and x == _BF16):
        raise TypeError("beside a stream of %s the block's values must be bfloat16%s, got %s" % (x, "" if x == _BF16 else " or float32", f))
    return f


def ra_norm_block(x, f=None, post=None, gate=None, alpha: float = 1.0, beta: float = 1.0, pre=None, dtype=None, out=None, h=None,
                  keep: bool = True, stream=None):
    """What lies between two blocks of a layer:
        x' = alpha * x + beta * gate * post(f),   h = pre(x')
    Returns (x', h, kept).  x [rows, d] is the residual stream, f the output of
    the block behind (None: x' is x itself and only pre is computed), h the input
    of the block ahead (None without `pre`), `post` and `pre` Norms or None, gate
    a vector of d values or a matrix like f.  pre is taken of x' as it is stored.

    The stream is float32 or bfloat16; f and h have one type, bfloat16 or the
    stream's (dtype: h's where there is no f, bfloat16 unless given).  `out` (x',
    may be x itself) and `h` are allocated unless given.  kept: the float32
    [rows, 4] moments that ra_norm_block_grad takes, None with keep=False."""
    rows, d = s = _shape(x, "x")
    dev = _device(x.get_device())
    px, ldx, xcode = _matrix(x, "x", dev, None, s)
    pf = ldf = po = ldo = pg = ldg = gkind = gcode = 0
    if f is not None:
        block = _block_type(f.dtype, x.dtype)
        if dtype is not None and dtype != block:
            raise TypeError("dtype must be that of f, %s, got %s" % (block, dtype))
        pf, ldf = _like(f, "f", dev, block, s)
        if gate is not None:
            pg, ldg, gkind, gcode = _gate(gate, dev, rows, d, f)
        if out is None:
            out = _new(x, x.dtype, stream)
        po, ldo = _like(out, "out", dev, x.dtype, s)
    else:
        if post is not None or gate is not None or out is not None:
            raise ValueError("post, gate and out need f")
        if pre is None:
            raise ValueError("give f, pre, or both")
        block = _block_type(dtype or (_BF16 if h is None else h.dtype), x.dtype)
        out = x
    ph = ldh = 0
    behind, ahead = _norm(post, "post", dev, d), _norm(pre, "pre", dev, d)
    if pre is not None:
        if h is None:
            h = _new(x if f is None else f, block, stream)
        ph, ldh = _like(h, "h", dev, block, s)
    elif h is not None:
        raise ValueError("h needs pre")
    pk, kept = 0, None
    if keep:
        kept = _empty((rows, 4), _F32, x.device, stream)
        pk = kept.data_ptr()
    args = _BLOCK.pack(rows, d, px, ldx, pf, ldf, pg, ldg, po, ldo, ph, ldh, pk, *behind, *ahead, xcode, _CODE[block], gkind, gcode, alpha, beta)
    _check(_load().ra_norm_block(args, _stream_of(stream, dev)), "ra_norm_block")
    return out, h, kept


class NormBlockGrads:
    """Gradients of ra_norm_block: dx and df (matrices), gate (a float32 vector,
    or a matrix like the gate), and post_gain, post_bias, pre_gain, pre_bias
    (float32 vectors).  What is None is not there, or not wanted."""

    __slots__ = ("dx", "df", "gate", "post_gain", "post_bias", "pre_gain", "pre_bias")

    def __init__(self, dx=None, df=None, gate=None, post_gain=None, post_bias=None, pre_gain=None, pre_bias=None):
        self.dx, self.df, self.gate = dx, df, gate
        self.post_gain, self.post_bias, self.pre_gain, self.pre_bias = post_gain, post_bias, pre_gain, pre_bias


def ra_norm_block_grad(dh, x, kept, f=None, post=None, gate=None, alpha: float = 1.0, beta: float = 1.0, pre=None, dx=None, out=None,
                       accumulate: bool = False, workspace=None, stream=None) -> NormBlockGrads:
    """The gradients of ra_norm_block, from dh (of h; None without `pre`) and dx
    (of x', what the later part of the stream sends back; None: zeros).

    x is x' as ra_norm_block returned it, kept its moments, and the rest what it
    was given.  Without `out` all gradients there are get computed: dx, df where
    there is an f, the gate's, and those of the gains and biases given.  `out`, a
    NormBlockGrads, holds the tensors to write instead, for views of a worker's
    flat gradient or fewer gradients; its dx may be the dx given.  accumulate adds
    to its vectors (micro-batches)."""
    rows, d = s = _shape(x, "x")
    stream_type = x.dtype
    dev = _device(x.get_device())
    px, ldx, xcode = _matrix(x, "x", dev, None, s)
    ph = ldh = pd = ldd = pf = ldf = pg = ldg = gkind = gcode = pk = 0
    block = None
    if f is not None:
        block = _block_type(f.dtype, stream_type)
        pf, ldf = _like(f, "f", dev, block, s)
        if gate is not None:
            pg, ldg, gkind, gcode = _gate(gate, dev, rows, d, f)
    elif post is not None or gate is not None:
        raise ValueError("post and gate need f")
    if (dh is None) != (pre is None):
        raise ValueError("dh and pre go together")
    if dh is not None:
        if block is None:
            block = _block_type(dh.dtype, stream_type)
        ph, ldh = _like(dh, "dh", dev, block, s)
    elif dx is None:
        raise ValueError("give dh, dx, or both")
    if dx is not None:
        pd, ldd = _like(dx, "dx", dev, stream_type, s)
    if pre is not None or post is not None:
        if kept is None or kept.dtype is not _F32 or kept.shape != (rows, 4) or kept.get_device() != dev or not kept.is_contiguous():
            raise ValueError("kept must be the float32 [%d, 4] tensor that ra_norm_block returned" % rows)
        pk = kept.data_ptr()
    behind, ahead = _norm(post, "post", dev, d), _norm(pre, "pre", dev, d)
    lib = _load()
    need = lib.ra_norm_block_grad_workspace_bytes(rows, d)
    po = ldo = pdf = lddf = pdg = lddg = pgg = pgb = prg = prb = pw = 0
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
        out = NormBlockGrads()
        out.dx = t = _new(x, stream_type, stream)
        po, ldo = t.data_ptr(), d
        if f is not None:
            out.df = t = _new(f, block, stream)
            pdf, lddf = t.data_ptr(), d
            if gkind == 2:
                out.gate = t = _new(gate, block, stream)
                pdg, lddg = t.data_ptr(), d
        # the vectors' gradients are rows of one small array
        count = (ahead[0] != 0) + (ahead[1] != 0) + (behind[0] != 0) + (behind[1] != 0) + (gkind == 1)
        if count:
            sums = _empty((count, d), _F32, x.device, stream)
            at, vectors = sums.data_ptr(), iter(sums.unbind())
            if ahead[0]:
                out.pre_gain, prg, at = next(vectors), at, at + 4 * d
            if ahead[1]:
                out.pre_bias, prb, at = next(vectors), at, at + 4 * d
            if behind[0]:
                out.post_gain, pgg, at = next(vectors), at, at + 4 * d
            if behind[1]:
                out.post_bias, pgb, at = next(vectors), at, at + 4 * d
            if gkind == 1:
                out.gate, pdg, lddg = next(vectors), at, d
    elif not isinstance(out, NormBlockGrads):
        raise TypeError("out must be a NormBlockGrads")
    else:
        if out.dx is not None:
            po, ldo = _like(out.dx, "out.dx", dev, stream_type, s)
        if out.df is not None:
            if f is None:
                raise ValueError("out.df needs f")
            pdf, lddf = _like(out.df, "out.df", dev, block, s)
        if out.gate is not None:
            if gkind == 0:
                raise ValueError("out.gate needs a gate")
            if gkind == 2:
                pdg, lddg = _like(out.gate, "out.gate", dev, block, s)
            else:
                pdg, lddg = _vector(out.gate, "out.gate", dev, d, _F32)[0], d
        if (out.post_gain is not None or out.post_bias is not None) and post is None:
            raise ValueError("out.post_gain and out.post_bias need post")
        if (out.pre_gain is not None or out.pre_bias is not None) and pre is None:
            raise ValueError("out.pre_gain and out.pre_bias need pre")
        pgg, pgb, prg, prb = (0 if t is None else _vector(t, what, dev, d, _F32)[0]
                              for t, what in ((out.post_gain, "out.post_gain"), (out.post_bias, "out.post_bias"), (out.pre_gain, "out.pre_gain"),
                                              (out.pre_bias, "out.pre_bias")))
        count = pgg or pgb or prg or prb or (gkind == 1 and pdg)
    on = _stream_of(stream, dev)
    hold = taken = None
    if count:
        if workspace is not None or not _raw_alloc or not need:
            hold, pw, need = _workspace(workspace, need, x, stream)
        else:
            pw = taken = _raw_alloc(need, on)
    try:
        args = _BLOCK_GRAD.pack(rows, d, ph, ldh, pd, ldd, px, ldx, pf, ldf, pg, ldg, pk, po, ldo, pdf, lddf, pdg, lddg, pgg, pgb, prg, prb, pw, need,
                                *behind, *ahead, xcode, xcode if block is None else _CODE[block], gkind, gcode, alpha, beta, int(accumulate), 0)
        _check(lib.ra_norm_block_grad(args, on), "ra_norm_block_grad")
    finally:
        if taken:  # the allocator gives it to later work of this stream
            _raw_delete(taken)
    return out


# ---------------------------------------------------------------------------
# log probabilities


class LogProbs:
    """What ra_logprobs returns for its rows: logp (of the given tokens), lse,
    entropy, top_ids and top_logp; None where not asked for."""

    __slots__ = ("logp", "lse", "entropy", "top_ids", "top_logp")

    def __init__(self, logp, lse, entropy, top_ids, top_logp):
        self.logp, self.lse, self.entropy, self.top_ids, self.top_logp = logp, lse, entropy, top_ids, top_logp


def ra_logprobs(logits, ids=None, scale: float = 1.0, entropy: bool = False, top: int = 0, stream=None) -> LogProbs:
    """Of softmax(scale * logits), row by row: the log probability of the row's
    token ids[r] (0 for an id outside the vocabulary, padding), the logarithm of
    the sum of exponentials, and if asked the entropy and the `top` most likely
    tokens (int64, -1 where no possible token is left) with their log
    probabilities, the lowest index first among equals.  A logit of minus
    infinity is a token that cannot be; a row with a NaN or plus infinity gives
    NaN.  All results but the tokens are float32."""
    rows, vocab = s = _shape(logits, "logits")
    dev = _device(logits.get_device())
    pz, ldz, code = _matrix(logits, "logits", dev, None, s)
    if not 0 <= top <= MAX_TOP:
        raise ValueError("top must lie between 0 and %d, got %r" % (MAX_TOP, top))
    pi, size, results = None, 8, 1 + (ids is not None) + bool(entropy)
    if ids is not None:
        pi, size, count = _ids(ids, dev)
        if count != rows:
            raise ValueError("give one id for each of the %d rows, got %d" % (rows, count))
    buffer = _empty((results + top, rows), _F32, logits.device, stream)
    lse = buffer[0]
    p = lse.data_ptr()
    logp = h = top_ids = top_logp = pl = ph = pt = pv = None
    if ids is not None:
        logp, pl = buffer[1], p + 4 * rows
    if entropy:
        h, ph = buffer[results - 1], p + 4 * rows * (results - 1)
    if top:
        top_logp = buffer[results:].view(rows, top)
        top_ids = _empty((rows, top), torch.int64, logits.device, stream)
        pt, pv = top_ids.data_ptr(), p + 4 * rows * results
    _check(_load().ra_logprobs(pz, ldz, code, rows, vocab, pi, size, scale, pl, p, ph, top, pt, pv, _stream_of(stream, dev)), "ra_logprobs")
    return LogProbs(logp, lse, h, top_ids, top_logp)


def ra_logprobs_grad(logits, ids, lse, grad_logp=None, scale: float = 1.0, entropy=None, grad_entropy=None, dtype=None, out=None, stream=None):
    """The gradient with respect to the logits, from those of ra_logprobs' logp
    and entropy (float32 vectors; None: zeros).  lse, and with grad_entropy also
    entropy, are what ra_logprobs returned.  dtype: the new output's type (the
    logits' unless given); `out` may be the logits themselves."""
    rows, vocab = s = _shape(logits, "logits")
    dev = _device(logits.get_device())
    pz, ldz, code = _matrix(logits, "logits", dev, None, s)
    pl, _ = _vector(lse, "lse", dev, rows, _F32)
    pi, size, pg, ph, pe = None, 8, None, None, None
    if grad_logp is not None:
        pg, _ = _vector(grad_logp, "grad_logp", dev, rows, _F32)
        pi, size, count = _ids(ids, dev)
        if count != rows:
            raise ValueError("give one id for each of the %d rows, got %d" % (rows, count))
    if grad_entropy is not None:
        if entropy is None:
            raise ValueError("grad_entropy needs entropy")
        pe, _ = _vector(grad_entropy, "grad_entropy", dev, rows, _F32)
        ph, _ = _vector(entropy, "entropy", dev, rows, _F32)
    out, po, ldo, ocode = _output(out, rows, vocab, dtype or (logits.dtype if out is None else None), logits, dev, stream)
    _check(_load().ra_logprobs_grad(pz, ldz, code, rows, vocab, pi, size, scale, pl, ph, pg, pe, po, ldo, ocode, _stream_of(stream, dev)),
           "ra_logprobs_grad")
    return out
