"""ra_norm_block and ra_norm_block_grad where binary32 ends, without rows, and what
the gradients keep alive."""
from __future__ import annotations

import pytest
import torch

import gradient_ring_all_gb300 as ra
from block_reference import CHAIN, _norm64, half_step, join64
from operator_reference import check

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


@pytest.mark.parametrize("d", [40, 1003, 2048, 8192, 16384])
def test_a_mean_whose_square_leaves_binary32(d):
    """The variance of such rows is that of the differences, behind a block and before one."""
    g = torch.Generator(device="cuda").manual_seed(d)
    x = torch.randn(5, d, generator=g, device="cuda") * 1e17 + torch.tensor([[3e19], [-3e19], [1e20], [2e19], [0.0]], device="cuda")
    n = ra.Norm(torch.randn(d, generator=g, device="cuda"), torch.randn(d, generator=g, device="cuda"))
    _, h, kept = ra.ra_norm_block(x, pre=n, dtype=F32)
    want, size, _, _, m, rstd = _norm64(x.double(), n)
    check(h, want, CHAIN * size, "h")
    check(kept[:, 3], rstd.squeeze(1), 2.0 ** -10 * rstd.squeeze(1), "rstd")  # the mean is off by 64 u of its size, 4e-3 of a deviation, and the variance by the square
    zero = torch.zeros(5, d, device="cuda")
    new, _, kept = ra.ra_norm_block(zero, x, post=n)
    want, size = join64(zero, x, n, None, 1.0, 1.0)
    check(new, want, CHAIN * size + half_step(F32) * want.abs(), "x'")
