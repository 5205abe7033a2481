"""What a Norm holds (no GPU)."""
from __future__ import annotations

import pytest


def test_a_norm_computes_the_kind_that_it_shows():
    pytest.importorskip("torch")
    from gradient_ring_all_gb300 import block_operators as b
    n = b.Norm(eps=1e-6)
    assert n.kind == "layer" and b._norm(n, "pre", 0, 8)[3] == 1
    n.kind = "rms"
    assert n.kind == "rms" and b._norm(n, "pre", 0, 8)[3] == 2
    with pytest.raises(ValueError, match="layer, rms"):
        n.kind = "batch"
    assert n.kind == "rms"
