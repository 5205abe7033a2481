"""ra_norm_block and ra_norm_block_grad where binary32 ends, without rows, and what
the gradients keep alive."""
from __future__ import annotations

import pytest
import torch

import gradient_ring_all_gb300 as ra

pytestmark = pytest.mark.gpu

F32 = torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from gradient_ring_all_gb300 import build
    build.build()
    ra.load()


@pytest.mark.parametrize("rows,d", [(3, 2048), (400, 24), (5, 4096)])
def test_gradients_do_not_hold_the_workspace(rows, d):
    x = torch.randn(rows, d, device="cuda")
    n = ra.Norm(torch.ones(d, device="cuda"), torch.zeros(d, device="cuda"))
    gate = torch.ones(d, device="cuda")
    new, h, kept = ra.ra_norm_block(x, x + 1, post=n, gate=gate, pre=n, dtype=F32)
    g = ra.ra_norm_block_grad(h, new, kept, f=x + 1, post=n, gate=gate, pre=n)
    for t in (g.pre_gain, g.pre_bias, g.post_gain, g.post_bias, g.gate):
        assert t.shape == (d,) and t.is_contiguous() and t.untyped_storage().nbytes() <= 5 * d * 4
