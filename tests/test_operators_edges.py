"""The operators on the host (no GPU): edges of what is accepted and refused.
No call here gets as far as a launch."""
from __future__ import annotations

import pytest

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


@pytest.mark.parametrize("act", [0, 1, 2, 3])
def test_weight_gradient_of_an_empty_checkpoint(lib, act):
    """An empty array has no address: both pointers of an empty checkpoint may be NULL."""
    def wgrad(m, k, n, q=None, e=None):
        return lib.ra_linear_wgrad(None, k, q, e, act, B, n, m, k, n, 0, C, n, F32, None, W, 1 << 24, None)

    assert wgrad(16, 0, 32) == OK and wgrad(0, 24, 0) == OK and wgrad(0, 0, 0) == OK
    # a checkpoint that has values is asked for
    assert wgrad(16, 24, 32) == INVALID and wgrad(16, 24, 32, q=D) == INVALID and wgrad(16, 24, 32, e=E) == INVALID


class _Elsewhere:
    """The look of a matrix on device 1."""

    def __init__(self, dtype, *shape):
        import torch
        self.shape, self.dtype = torch.Size(shape), dtype

    def get_device(self):
        return 1

    def stride(self):
        return self.shape[1], 1

    def is_contiguous(self):
        return True

    def numel(self):
        return self.shape.numel()

    def data_ptr(self):
        raise AssertionError("looked at an address on another device")


def test_tensors_on_another_device_than_the_current_one_are_refused(monkeypatch):
    """The library launches on the current device, whatever device the addresses belong to."""
    torch = pytest.importorskip("torch")
    from gradient_ring_all_gb300 import operators as op
    monkeypatch.setattr(op, "_current_device", lambda: 0, raising=False)
    x, w, ids = _Elsewhere(torch.bfloat16, 4, 8), _Elsewhere(torch.bfloat16, 8, 8), _Elsewhere(torch.int64, 4)
    kept = object.__new__(op.Checkpoint8)
    kept.rows, kept.cols, kept._dev, kept._pq, kept._pe = 4, 8, 1, 0, 0
    for call in (lambda: op.ra_checkpoint8_pack(x), lambda: op.ra_checkpoint8_unpack(kept, out=x), lambda: op.ra_embedding_lookup(x, ids, out=x),
                 lambda: op.ra_embedding_grad(x, ids, 4, out=x), lambda: op.ra_linear(x, w, out=x), lambda: op.ra_linear_dgrad(x, w, out=x),
                 lambda: op.ra_linear_wgrad(x, x, out=w)):
        with pytest.raises(ValueError, match="cuda:1"):
            call()


def test_column_slices_side_by_side(lib):
    """x and y as column slices of one array: side by side they are fine (the call then asks for the workspace that rows 57
    values apart need), a column into each other they overlap; so do slices of arrays with another stride."""
    def linear(at, ld=57):
        return lib.ra_linear(A, 57, B, 32, 16, 24, 32, None, F32, 0, None, 0, F32, None, None, A + 2 * at, ld, BF16, None, 0, None)

    assert linear(24) == INVALID and linear(25) == INVALID
    assert linear(23) == OVERLAP and linear(26) == OVERLAP  # into x's columns; into those of x's next row
    assert linear(24, 58) == OVERLAP


def test_a_single_row_between_another_matrix_rows(lib):
    """A vector, or one row, in the gap between the rows of an output shares no byte with it (the call then asks for the
    workspace that rows 57 values apart need); one that reaches into the next row does."""
    def linear(bias, n=32, ldy=100):
        return lib.ra_linear(A, 57, B, n, 16, 24, n, bias, BF16, 0, None, 0, F32, None, None, C, ldy, BF16, None, 0, None)

    assert linear(C + 2 * 32) == INVALID and linear(C + 2 * 68) == INVALID and linear(C + 2 * 332) == INVALID
    assert linear(C + 2 * 31) == OVERLAP and linear(C + 2 * 69) == OVERLAP and linear(C) == OVERLAP and linear(C + 2 * 100) == OVERLAP
    # in front of the first row and behind the last one it is elsewhere
    assert linear(C - 2 * 32) == INVALID and linear(C + 2 * (15 * 100 + 32)) == INVALID
    assert linear(C - 2 * 31) == OVERLAP and linear(C + 2 * (15 * 100 + 31)) == OVERLAP
    # a row as long as the distance of the other's rows or longer fits no gap
    assert linear(C + 2 * 64, n=64, ldy=100) == OVERLAP


def test_workspace_of_sizes_that_no_call_takes(lib):
    """Matrices past 2^46 bytes are refused by the calls; the questions about their workspaces answer 0."""
    big = (1 << 31) - 1
    for m, k, n in ((big, big, 1), (1, big, big), (big, 1, big), (big, big, big), (1 << 23, 1 << 23, 8)):
        assert lib.ra_linear_workspace_bytes(m, k, n) == 0
    assert lib.ra_linear(A, big, B, 1, big, big, 1, None, F32, 0, None, 0, F32, None, None, C, 1, BF16, W, 1 << 24, None) == INVALID
    # the largest that is taken: two matrices laid out, rows of whole 32 bytes
    assert lib.ra_linear_workspace_bytes(1 << 22, 1 << 22, 7) == (1 << 45) + (1 << 22) * 32 + 32
    assert lib.ra_linear_workspace_bytes(5, 7, 9) == 2 * 256 + 32
