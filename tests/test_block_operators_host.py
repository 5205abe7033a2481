"""The operators between a step's products on the host (no GPU): bad arguments
are refused before anything is queued, sizes of zero are no-ops, and the binding
packs what the header declares.  No call here gets as far as a launch."""
from __future__ import annotations

import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, OVERLAP = 0, 1, 2, 3
F32, BF16 = 0, 1
NONE, LAYER, RMS = 0, 1, 2
A, B, C, D, E, F, G, H, W = (0x10000000 * k for k in range(1, 10))  # far apart, never touched


@pytest.fixture(scope="module")
def lib():
    pytest.importorskip("torch")
    from gradient_ring_all_gb300 import build
    build.build()
    from gradient_ring_all_gb300 import block_operators
    return block_operators._load()


def test_the_generator_of_the_reference():
    """Known answers of Philox4x32-10 (published with its paper), and the array form against the plain one."""
    pytest.importorskip("torch")
    from block_reference import keep_mask, philox
    assert philox((0, 0, 0, 0), (0, 0)) == [0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8]
    assert philox((2 ** 32 - 1,) * 4, (2 ** 32 - 1,) * 2) == [0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd]
    assert philox((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0)) == [0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1]
    seed, first = (5 << 32) + 77, (3 << 32) - 1
    mask = keep_mask(2, 19, 0.3, seed, 9, first)
    for r in range(2):
        for c in range(19):
            word = philox((c // 8, 9, (first + r) % 2 ** 32, (first + r) >> 32), (77, 5))[c % 8 // 2]
            assert bool(mask[r, c]) == ((word >> 16 * (c % 2)) & 0xFFFF >= round(65536 * 0.3))


def test_dropout(lib):
    def drop(x=A, ldx=24, xt=BF16, rows=16, cols=24, p=0.5, seed=1, at=None, first=0, r=None, ldr=24, rt=BF16, y=C, ldy=24, yt=BF16):
        return lib.ra_dropout(x, ldx, xt, rows, cols, p, seed, at, 0, first, r, ldr, rt, y, ldy, yt, None)

    assert drop(x=None) == INVALID and drop(y=None) == INVALID and drop(xt=2) == INVALID and drop(yt=-1) == INVALID and drop(r=B, rt=9) == INVALID
    assert drop(p=-0.001) == INVALID and drop(p=1.001) == INVALID and drop(p=float("nan")) == INVALID
    assert drop(ldx=23) == INVALID and drop(ldy=23) == INVALID and drop(r=B, ldr=23) == INVALID and drop(x=A + 1) == INVALID and drop(r=B + 1) == INVALID
    assert drop(at=D + 4) == INVALID and drop(first=-1) == INVALID and drop(first=2 ** 63 - 8) == INVALID
    assert drop(rows=-1) == INVALID and drop(cols=-1) == INVALID and drop(rows=1 << 31) == INVALID
    assert drop(y=A + 2) == OVERLAP and drop(y=A, yt=F32) == OVERLAP and drop(y=A, ldy=25) == OVERLAP
    assert drop(r=C + 2) == OVERLAP and drop(r=C, rt=F32) == OVERLAP and drop(at=C + 8) == OVERLAP
    assert drop(rows=0) == OK and drop(cols=0) == OK and drop(cols=0, x=None, y=None) == OK


class _Norm(ctypes.Structure):
    _fields_ = [("gain", ctypes.c_void_p), ("bias", ctypes.c_void_p), ("dtype", ctypes.c_int), ("kind", ctypes.c_int), ("eps", ctypes.c_float),
                ("reserved", ctypes.c_int)]


def _matrices(*names):
    return [f for n in names for f in ((n, ctypes.c_void_p), ("ld_" + n, ctypes.c_int64))]


_TYPES = [("post", _Norm), ("pre", _Norm), ("x_dtype", ctypes.c_int), ("f_dtype", ctypes.c_int), ("gate_kind", ctypes.c_int), ("gate_dtype", ctypes.c_int),
          ("alpha", ctypes.c_float), ("beta", ctypes.c_float)]


class _Block(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("d", ctypes.c_int64)] + _matrices("x", "f", "gate", "x_out", "h") + [("kept", ctypes.c_void_p)] + _TYPES


class _Grad(ctypes.Structure):
    _fields_ = ([("rows", ctypes.c_int64), ("d", ctypes.c_int64)] + _matrices("dh", "dx_new", "x", "f", "gate") + [("kept", ctypes.c_void_p)]
                + _matrices("dx", "df", "dgate") + [(n, ctypes.c_void_p) for n in ("dpost_gain", "dpost_bias", "dpre_gain", "dpre_bias", "ws")]
                + [("ws_bytes", ctypes.c_size_t)] + _TYPES + [("accumulate", ctypes.c_int), ("reserved", ctypes.c_int)])


def _norm(kind=LAYER, gain=G, bias=None, dtype=F32, eps=1e-5, reserved=0):
    return _Norm(gain, bias, dtype, kind, eps, reserved)


def test_norm_block(lib):
    def block(**kw):
        rows, d = kw.pop("rows", 16), kw.pop("d", 24)
        a = _Block(rows=rows, d=d, x=A, ld_x=24, f=B, ld_f=24, gate=None, ld_gate=24, x_out=C, ld_x_out=24, h=D, ld_h=24, kept=E, post=_norm(),
                   pre=_norm(RMS), x_dtype=BF16, f_dtype=BF16, gate_kind=0, gate_dtype=F32, alpha=1, beta=1)
        for k, v in kw.items():
            setattr(a, k, v)
        return lib.ra_norm_block(ctypes.string_at(ctypes.byref(a), ctypes.sizeof(a)), None)

    assert lib.ra_norm_block(None, None) == INVALID
    for name in ("x", "x_out", "h"):
        assert block(**{name: None}) == INVALID, name
        assert block(**{name: A + 1 if name == "x" else F + 1}) == INVALID, name
    for name in ("ld_x", "ld_f", "ld_x_out", "ld_h"):
        assert block(**{name: 23}) == INVALID, name
    assert block(x_dtype=2) == INVALID and block(f_dtype=2) == INVALID and block(f_dtype=F32) == INVALID  # a bf16 stream's block is bf16
    assert block(post=_norm(3)) == INVALID and block(pre=_norm(-1)) == INVALID and block(pre=_norm(eps=-1.0)) == INVALID
    assert block(pre=_norm(eps=float("nan"))) == INVALID and block(pre=_norm(dtype=5)) == INVALID and block(pre=_norm(reserved=1)) == INVALID
    assert block(post=_norm(gain=G + 2)) == INVALID and block(post=_norm(bias=G + 1, dtype=BF16)) == INVALID
    assert block(gate_kind=1) == INVALID and block(gate_kind=3, gate=H) == INVALID and block(gate_kind=1, gate=H, gate_dtype=4) == INVALID
    assert block(gate_kind=2, gate=H, ld_gate=23) == INVALID and block(kept=E + 8) == INVALID
    assert block(rows=-1) == INVALID and block(d=-1) == INVALID
    assert block(f=None, pre=_norm(NONE)) == INVALID
    big = 32769
    assert block(d=big, ld_x=big, ld_f=big, ld_x_out=big, ld_h=big) == UNSUPPORTED
    for name in ("x_out", "h", "kept"):
        for at in (A + 32, B + 32, G):
            assert block(**{name: at}) == OVERLAP, (name, at)
    assert block(h=C) == OVERLAP and block(kept=C) == OVERLAP and block(kept=D + 32) == OVERLAP and block(x_out=A, ld_x_out=25) == OVERLAP
    assert block(gate_kind=1, gate=C + 64) == OVERLAP and block(gate_kind=2, gate=D + 64) == OVERLAP
    assert block(rows=0) == OK and block(d=0) == OK


def test_norm_block_grad(lib):
    need = lib.ra_norm_block_grad_workspace_bytes(16, 24)
    assert need > 0 and lib.ra_norm_block_grad_workspace_bytes(0, 24) == 0 and lib.ra_norm_block_grad_workspace_bytes(16, 32769) == 0
    assert lib.ra_norm_block_grad_workspace_bytes(1 << 30, 32768) <= 152 * 5 * 32768 * 4

    def grad(**kw):
        a = _Grad(rows=16, d=24, dh=A, ld_dh=24, dx_new=B, ld_dx_new=24, x=C, ld_x=24, f=D, ld_f=24, gate=None, ld_gate=24, kept=E, dx=F, ld_dx=24, df=H,
                  ld_df=24, dgate=None, ld_dgate=24, dpost_gain=H + 0x100000, dpost_bias=H + 0x200000, dpre_gain=H + 0x300000, dpre_bias=H + 0x400000, ws=W,
                  ws_bytes=need, post=_norm(), pre=_norm(RMS), x_dtype=BF16, f_dtype=BF16, gate_kind=0, gate_dtype=F32, alpha=1, beta=1)
        for k, v in kw.items():
            setattr(a, k, v)
        return lib.ra_norm_block_grad(ctypes.string_at(ctypes.byref(a), ctypes.sizeof(a)), None)

    assert lib.ra_norm_block_grad(None, None) == INVALID
    for name in ("dh", "x", "kept", "ws"):
        assert grad(**{name: None}) == INVALID, name
    for name in ("ld_dh", "ld_dx_new", "ld_x", "ld_f", "ld_dx", "ld_df"):
        assert grad(**{name: 23}) == INVALID, name
    for name in ("dpost_gain", "dpost_bias", "dpre_gain", "dpre_bias"):
        assert grad(**{name: H + 0x500002}) == INVALID, name
        assert grad(**{name: F + 64}) == OVERLAP and grad(**{name: A + 64}) == OVERLAP and grad(**{name: G}) == OVERLAP, name
    assert grad(ws_bytes=need - 1) == INVALID and grad(ws=W + 8) == INVALID and grad(kept=E + 8) == INVALID and grad(reserved=1) == INVALID
    assert grad(x_dtype=3) == INVALID and grad(f_dtype=F32) == INVALID and grad(pre=_norm(7)) == INVALID
    # what is not there has no gradient
    assert grad(f=None) == INVALID and grad(f=None, df=None) == INVALID and grad(pre=_norm(NONE)) == INVALID and grad(post=_norm(NONE)) == INVALID
    assert grad(dgate=H + 0x600000) == INVALID and grad(pre=_norm(NONE), dh=None, dx_new=None, dpre_gain=None, dpre_bias=None) == INVALID
    for name in ("dx", "df"):
        for at in (A, C + 64, D + 64, E, G):
            assert grad(**{name: at}) == OVERLAP, (name, at)
    assert grad(dx=B + 48) == OVERLAP and grad(dx=B, ld_dx=25) == OVERLAP and grad(df=B) == OVERLAP and grad(df=F) == OVERLAP
    assert grad(ws=A) == OVERLAP and grad(ws=F) == OVERLAP and grad(dpre_bias=H + 0x300000) == OVERLAP
    gates = dict(gate=H + 0x700000, gate_kind=1)
    assert grad(dgate=H + 0x700000, **gates) == OVERLAP and grad(dgate=H + 0x600002, **gates) == INVALID and grad(gate_dtype=7, **gates) == INVALID
    assert grad(d=0) == OK
    big = 32769
    assert grad(d=big, **{"ld_" + n: big for n in ("dh", "dx_new", "x", "f", "dx", "df")}) == UNSUPPORTED


def test_logprobs(lib):
    def logp(z=A, ld=24, t=BF16, rows=16, vocab=24, ids=B, ib=8, scale=1.0, lp=C, lse=D, h=E, top=3, ti=F, tv=H):
        return lib.ra_logprobs(z, ld, t, rows, vocab, ids, ib, scale, lp, lse, h, top, ti, tv, None)

    assert logp(z=None) == INVALID and logp(ids=None) == INVALID and logp(lse=None) == INVALID and logp(ti=None) == INVALID and logp(tv=None) == INVALID
    assert logp(t=2) == INVALID and logp(ld=23) == INVALID and logp(ib=2) == INVALID and logp(ids=B + 4) == INVALID and logp(z=A + 1) == INVALID
    for bad in (0.0, -1.0, float("nan"), float("inf"), 3e38):
        assert logp(scale=bad) == INVALID
    assert logp(top=-1) == INVALID and logp(top=33) == INVALID and logp(lp=C + 2) == INVALID and logp(ti=F + 4) == INVALID and logp(tv=H + 2) == INVALID
    assert logp(rows=-1) == INVALID and logp(vocab=-1) == INVALID and logp(rows=1 << 31) == INVALID and logp(vocab=1 << 31) == INVALID
    for kw in (dict(lp=A), dict(lse=B + 8), dict(h=D), dict(ti=A + 64), dict(tv=F), dict(lp=E + 4)):
        assert logp(**kw) == OVERLAP, kw
    assert logp(rows=0) == OK

    def grad(z=A, ld=24, t=BF16, rows=16, vocab=24, ids=B, ib=8, scale=1.0, lse=C, h=D, g=E, gh=F, out=H, ldo=24, ot=BF16):
        return lib.ra_logprobs_grad(z, ld, t, rows, vocab, ids, ib, scale, lse, h, g, gh, out, ldo, ot, None)

    assert grad(z=None) == INVALID and grad(ids=None) == INVALID and grad(lse=None) == INVALID and grad(h=None) == INVALID and grad(out=None) == INVALID
    assert grad(t=2) == INVALID and grad(ot=2) == INVALID and grad(ib=1) == INVALID and grad(ldo=23) == INVALID and grad(scale=0.0) == INVALID
    assert grad(g=E + 2) == INVALID and grad(gh=F + 1) == INVALID
    for kw in (dict(out=A + 64), dict(out=A, ot=F32), dict(out=A, ldo=25), dict(out=B), dict(out=C), dict(out=D), dict(out=E), dict(out=F)):
        assert grad(**kw) == OVERLAP, kw
    assert grad(rows=0) == OK and grad(vocab=0) == OK


def test_the_binding_packs_what_the_header_declares(tmp_path):
    pytest.importorskip("torch")
    from gradient_ring_all_gb300 import block_operators as b
    src, exe = tmp_path / "s.c", tmp_path / "s"
    src.write_text('#include <stdio.h>\n#include "ra_operators.h"\nint main(void) { printf("%d %d %d\\n", (int)sizeof(ra_norm), '
                   "(int)sizeof(ra_norm_block_args), (int)sizeof(ra_norm_block_grad_args)); return 0; }\n")
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    sizes = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert sizes == [ctypes.sizeof(_Norm), ctypes.sizeof(_Block), ctypes.sizeof(_Grad)] == [32, b._BLOCK.size, b._BLOCK_GRAD.size]


def test_binding_refuses_before_the_library():
    torch = pytest.importorskip("torch")
    import gradient_ring_all_gb300 as ra
    t, i = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int64)
    kept = torch.zeros(4, 4)
    for call in (lambda: ra.ra_dropout(t, 0.5, 1), lambda: ra.ra_norm_block(t, pre=ra.Norm()), lambda: ra.ra_norm_block_grad(t, t, kept, pre=ra.Norm()),
                 lambda: ra.ra_logprobs(t, i), lambda: ra.ra_logprobs_grad(t, i, t[:, 0], t[:, 0]), lambda: ra.Norm(kind="batch"),
                 lambda: ra.Norm(eps=-1.0), lambda: ra.ra_dropout(t[0], 0.5, 1)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        ra.ra_logprobs(i.view(2, 2))


class _Elsewhere:
    """The look of a matrix on device 1."""

    def __init__(self, dtype, *shape):
        import torch
        self.shape, self.dtype = torch.Size(shape), dtype

    def get_device(self):
        return 1

    def stride(self):
        return self.shape[1], 1

    def data_ptr(self):
        raise AssertionError("looked at an address on another device")


def test_tensors_on_another_device_than_the_current_one_are_refused(monkeypatch):
    torch = pytest.importorskip("torch")
    from gradient_ring_all_gb300 import block_operators as b
    from gradient_ring_all_gb300 import operators as op
    monkeypatch.setattr(op, "_current_device", lambda: 0, raising=False)
    x = _Elsewhere(torch.bfloat16, 4, 8)
    for call in (lambda: b.ra_dropout(x, 0.5, 1), lambda: b.ra_norm_block(x, x, pre=b.Norm()), lambda: b.ra_norm_block_grad(x, x, None, pre=b.Norm()),
                 lambda: b.ra_logprobs(x), lambda: b.ra_logprobs_grad(x, None, None)):
        with pytest.raises(ValueError, match="cuda:1"):
            call()
