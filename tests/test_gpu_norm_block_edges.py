"""ra_norm_block and ra_norm_block_grad where binary32 ends, without rows, and what
the gradients keep alive."""
from __future__ import annotations

import pytest
import torch

import gradient_ring_all_gb300 as ra
from block_reference import CHAIN, _norm64, grads64, half_step, join64
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


@pytest.mark.parametrize("d", [8, 16, 64])
def test_even_rows_of_huge_values(d):
    """m rstd is no binary32 number in a row of equal values of 2^120: what lies beside the row's end must not enter its sums."""
    x = torch.full((3, d), 2.0 ** 120, device="cuda")
    x[1] = torch.randn(d, device="cuda")
    n = ra.Norm(torch.randn(d, device="cuda"), torch.randn(d, device="cuda"))
    _, h, kept = ra.ra_norm_block(x, pre=n, dtype=F32)
    assert kept[0, 2] == 2.0 ** 120 and torch.equal(h[0], n.bias)
    dh = torch.randn(3, d, device="cuda")
    got = ra.ra_norm_block_grad(dh, x, kept, pre=n)
    want = grads64(dh, x, None, None, None, 1.0, 1.0, n, None)
    # the huge rows' normed values are 0, so their part of the magnitudes is that of a row of zeros
    small = x.clone()
    small[0], small[2] = 0.0, 0.0
    size = grads64(dh, small, None, None, None, 1.0, 1.0, n, None)
    check(got.dx, want["dx"][0], CHAIN * size["dx"][1] + half_step(F32) * want["dx"][0].abs(), "dx")
    check(got.pre_gain, want["pre_gain"][0], CHAIN * size["pre_gain"][1], "pre_gain")
    zero = torch.zeros(3, d, device="cuda")
    new, _, kept = ra.ra_norm_block(zero, x, post=n)
    got = ra.ra_norm_block_grad(None, new, kept, f=x, post=n, dx=dh)
    want = grads64(None, new, x, n, None, 1.0, 1.0, None, dh)
    size = grads64(None, new, small, n, None, 1.0, 1.0, None, dh)
    check(got.df, want["df"][0], CHAIN * size["df"][1] + half_step(F32) * want["df"][0].abs(), "df")
    check(got.post_gain, want["post_gain"][0], CHAIN * size["post_gain"][1], "post_gain")


def test_no_rows_beside_parameters_that_are_not_finite():
    """A sum over no rows is 0, whatever it would be multiplied with."""
    d = 24
    x = torch.zeros(0, d, device="cuda")
    odd = torch.full((d,), float("inf"), device="cuda")
    odd[3] = float("nan")
    n = ra.Norm(odd, odd)
    new, h, kept = ra.ra_norm_block(x, x, post=n, gate=odd, pre=n, dtype=F32)
    g = ra.ra_norm_block_grad(h, new, kept, f=x, post=n, gate=odd, pre=n)
    for t in (g.pre_gain, g.pre_bias, g.post_gain, g.post_bias, g.gate):
        assert not bool(t.any()) and not bool(torch.isnan(t).any())
    out = ra.NormBlockGrads(gate=torch.ones(d, device="cuda"), post_gain=torch.full((d,), 2.0, device="cuda"))
    ra.ra_norm_block_grad(h, new, kept, f=x, post=n, gate=odd, pre=n, out=out, accumulate=True)
    assert bool((out.gate == 1).all()) and bool((out.post_gain == 2).all())
