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
