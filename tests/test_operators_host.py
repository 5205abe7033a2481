"""The operators' C ABI on the host (no GPU): bad arguments are refused before
anything is queued, sizes of zero are no-ops, and the header is C."""
from __future__ import annotations

import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, OVERLAP = 0, 1, 2, 3
F32, BF16 = 0, 1
A, B, C, D, E, W = (0x10000000 * k for k in range(1, 7))  # far apart, never touched


@pytest.fixture(scope="module")
def lib():
    pytest.importorskip("torch")
    from gradient_ring_all_gb300 import build
    build.build()
    from gradient_ring_all_gb300 import operators
    return operators._load()


def test_checkpoint(lib):
    pack = lambda x=A, ld=64, t=F32, r=4, c=64, q=B, e=C: lib.ra_checkpoint8_pack(x, ld, t, r, c, q, e, None)  # noqa: E731
    assert pack(x=None) == INVALID and pack(q=None) == INVALID and pack(e=None) == INVALID
    assert pack(t=2) == INVALID and pack(ld=63) == INVALID and pack(x=A + 2) == INVALID and pack(q=B + 8) == INVALID
    assert pack(r=-1) == INVALID and pack(c=-1) == INVALID and pack(r=1 << 31) == INVALID
    assert pack(ld=1 << 60) == INVALID
    assert pack(q=A + 512) == OVERLAP and pack(e=A) == OVERLAP and pack(e=B + 255) == OVERLAP
    assert pack(r=0) == OK and pack(c=0, x=None, q=None, e=None) == OK
    un = lambda act=0, o=A, ld=64: lib.ra_checkpoint8_unpack(B, C, 4, 64, act, o, ld, BF16, None)  # noqa: E731
    assert un(act=4) == INVALID and un(act=-1) == INVALID and un(o=None) == INVALID and un(o=B) == OVERLAP


def test_embedding(lib):
    look = lambda t=A, ld=8, dt=F32, v=9, d=8, i=B, ib=8, n=5, o=C, lo=8: lib.ra_embedding_lookup(t, ld, dt, v, d, i, ib, n, 1.0, o, lo, None)  # noqa: E731
    assert look(t=None) == INVALID and look(i=None) == INVALID and look(o=None) == INVALID and look(ib=2) == INVALID
    assert look(dt=5) == INVALID and look(ld=7) == INVALID and look(lo=7) == INVALID and look(i=B + 4) == INVALID
    assert look(n=-1) == INVALID and look(o=A + 32) == OVERLAP and look(o=B) == OVERLAP
    assert look(n=0) == OK and look(d=0) == OK
    need = lib.ra_embedding_grad_workspace_bytes(5, 9, 8)
    assert need > 0 and lib.ra_embedding_grad_workspace_bytes(0, 9, 8) == 0
    grad = lambda g=A, gt=F32, i=B, ib=4, n=5, acc=0, o=C, ot=F32, v=9, d=8, w=W, nw=need: lib.ra_embedding_grad(  # noqa: E731
        g, d, gt, i, ib, n, 1.0, acc, o, d, ot, v, d, w, nw, None)
    assert grad(g=None) == INVALID and grad(i=None) == INVALID and grad(o=None) == INVALID and grad(w=None) == INVALID
    assert grad(nw=need - 1) == INVALID and grad(w=W + 8) == INVALID and grad(gt=3) == INVALID and grad(ot=-1) == INVALID
    assert grad(o=A) == OVERLAP and grad(o=B) == OVERLAP and grad(w=A) == OVERLAP and grad(w=C) == OVERLAP and grad(w=B) == OVERLAP
    assert grad(v=0) == OK and grad(n=0, acc=1, g=None, i=None, w=None, nw=0) == OK


def test_linear(lib):
    big = 1 << 24

    def lin(x=A, ldx=24, w=B, ldw=32, m=16, k=24, n=32, b=None, bt=F32, act=0, r=None, ldr=32, rt=BF16, q=None, e=None, y=C, ldy=32, yt=BF16):
        return lib.ra_linear(x, ldx, w, ldw, m, k, n, b, bt, act, r, ldr, rt, q, e, y, ldy, yt, W, big, None)

    assert lin(x=None) == INVALID and lin(w=None) == INVALID and lin(y=None) == INVALID
    assert lin(act=9) == INVALID and lin(yt=7) == INVALID and lin(b=D, bt=7) == INVALID and lin(r=D, rt=7) == INVALID
    assert lin(ldx=23) == INVALID and lin(ldw=31) == INVALID and lin(ldy=31) == INVALID and lin(r=D, ldr=31) == INVALID
    assert lin(m=-1) == INVALID and lin(x=A + 1) == INVALID and lin(q=D) == INVALID and lin(e=D) == INVALID and lin(q=D + 1, e=E) == INVALID
    assert lin(y=A) == OVERLAP and lin(y=B + 64) == OVERLAP and lin(b=C) == OVERLAP and lin(r=C + 64) == OVERLAP
    assert lin(r=C, rt=F32) == OVERLAP  # the residual in place has the output's type
    assert lin(q=A, e=E) == OVERLAP and lin(q=D, e=C) == OVERLAP and lin(q=D, e=D) == OVERLAP
    assert lin(m=0) == OK and lin(n=0) == OK

    def dgrad(dy=A, w=B, m=16, k=24, n=32, q=D, e=E, act=2, r=None, dx=C, xt=BF16):
        return lib.ra_linear_dgrad(dy, n, w, n, m, k, n, q, e, act, r, k, BF16, dx, k, xt, W, big, None)

    assert dgrad(dy=None) == INVALID and dgrad(w=None) == INVALID and dgrad(dx=None) == INVALID and dgrad(q=None) == INVALID
    assert dgrad(e=None) == INVALID and dgrad(act=4) == INVALID and dgrad(xt=2) == INVALID
    assert dgrad(dx=A) == OVERLAP and dgrad(dx=B) == OVERLAP and dgrad(dx=D) == OVERLAP and dgrad(r=C + 48) == OVERLAP
    assert dgrad(m=0) == OK and dgrad(k=0) == OK

    def wgrad(x=A, q=None, e=None, act=0, dy=B, m=16, k=24, n=32, dw=C, wt=F32, db=D):
        return lib.ra_linear_wgrad(x, k, q, e, act, dy, n, m, k, n, 0, dw, n, wt, db, W, big, None)

    assert wgrad(x=None) == INVALID and wgrad(dy=None) == INVALID and wgrad(dw=None) == INVALID and wgrad(act=1) == INVALID
    assert wgrad(q=E, e=E) == INVALID and wgrad(x=None, q=E) == INVALID and wgrad(wt=3) == INVALID and wgrad(db=D + 2) == INVALID
    assert wgrad(dw=A) == OVERLAP and wgrad(db=C) == OVERLAP and wgrad(db=B) == OVERLAP
    assert wgrad(x=None, q=C, e=E, act=1) == OVERLAP
    assert wgrad(k=0, db=None) == OK and wgrad(n=0) == OK


def test_column_slices_of_one_array_do_not_overlap(lib):
    # x and y as columns 0-23 and 24-55 of one array: reaches the workspace check, not the overlap check
    r = lib.ra_linear(A, 57, B, 32, 16, 24, 32, None, 0, 0, None, 0, 0, None, None, A + 2 * 23, 57, BF16, None, 0, None)
    assert r == OVERLAP  # one column too early


PROGRAM = r"""
#include <stdio.h>
#include "ra_operators.h"
int main(void) {
    ra_status a = ra_linear(0, 0, 0, 0, 1, 1, 1, 0, RA_F32, RA_ACT_GELU, 0, 0, RA_F32, 0, 0, 0, 0, RA_BF16, 0, 0, 0);
    ra_status b = ra_checkpoint8_pack(0, 0, RA_F32, 0, RA_CHECKPOINT8_GROUP, 0, 0, 0);
    printf("%d %d\n", (int)a, (int)b);
    return 0;
}
"""


def test_the_header_is_c_and_links(lib, tmp_path):
    src, exe = tmp_path / "ops.c", tmp_path / "ops"
    src.write_text(PROGRAM)
    libdir = os.path.join(ROOT, "gradient_ring_all_gb300", "lib")
    r = subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I", os.path.join(ROOT, "include"), str(src),
                        "-o", str(exe), "-L", libdir, "-lgradient_ring_all", "-Wl,-rpath," + libdir], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert out.stdout.split() == ["1", "0"]


def test_binding_refuses_before_the_library():
    torch = pytest.importorskip("torch")
    import gradient_ring_all_gb300 as ra
    t, i = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int64)
    for call in (lambda: ra.ra_embedding_lookup(t, i), lambda: ra.ra_embedding_grad(t, i, 4), lambda: ra.ra_checkpoint8_pack(t),
                 lambda: ra.ra_linear(t.bfloat16(), t.bfloat16().t()), lambda: ra.ra_linear_wgrad(t.bfloat16(), t.bfloat16())):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        ra.ra_checkpoint8_unpack(t)
    with pytest.raises(AttributeError):
        ra.no_such_call
