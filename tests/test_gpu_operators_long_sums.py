"""Products over long sums: the tensor core adds by truncation, always toward
zero, which must not show in a result.

The bound of the mean error.  With factors spread over a binade in every row and
column the results' places between two bf16 values are spread too, so a
rounding is off by up to half a step either way: 2^-8 / sqrt(12) = 1.13e-3 of the
value at most in the root mean square, and its mean over 128 x 128 results is within six times
1.13e-3 / 128 = 5.3e-5 of zero.  The sums' own error is below 1e-5: chunks of 512 are added by
up to 200 additions that round to nearest, and what a chunk loses is below 2e-6."""
from __future__ import annotations

import pytest
import torch

import gradient_ring_all_gb300 as ra
from operator_reference import act64, check, rounding, slope64, sum_bound, values64

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
MEAN = 6 * 1.13e-3 / 128 + 1e-5


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from gradient_ring_all_gb300 import build
    build.build()
    ra.load()


def _normal(seed, *shape, dtype=BF16, s=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * s).to(dtype)


def _positive(seed, k, cols):
    """k x cols values between 1 and 4; a column's share a factor of 1 to 2"""
    g = torch.Generator(device="cuda").manual_seed(seed)
    return ((1 + torch.rand(k, cols, generator=g, device="cuda")) * (1 + torch.rand(cols, generator=g, device="cuda"))).to(BF16)


@pytest.mark.parametrize("out_type", [BF16, F32])
@pytest.mark.parametrize("k", [16_400, 100_000])
@pytest.mark.parametrize("product", ["forward", "dgrad", "wgrad"])
def test_sums_of_one_sign_are_not_short(product, k, out_type):
    a, b = _positive(1, k, 2000), _positive(2, k, 2000)
    if product == "forward":
        got = ra.ra_linear(a.t().contiguous(), b, dtype=out_type)
    elif product == "dgrad":
        got = ra.ra_linear_dgrad(a.t().contiguous(), b.t().contiguous(), dtype=out_type)
    else:
        got = ra.ra_linear_wgrad(a, b, dtype=out_type)
    rows, cols = slice(0, 2000, 15), slice(0, 2000, 15)  # 134 x 134 of them
    want = torch.zeros(134, 134, dtype=torch.float64, device="cuda")
    for at in range(0, k, 8192):
        want += a[at:at + 8192, rows].double().t() @ b[at:at + 8192, cols].double()
    off = got[rows, cols].double() / want - 1
    assert abs(float(off.mean())) < (MEAN if out_type == BF16 else 1e-5)
    assert float(off.abs().max()) < (2.0 ** -8 if out_type == BF16 else 2e-5)


def test_sums_of_one_sign_below_the_length_that_is_made_in_chunks():
    """Up to 16384 of k a bf16 result may be short by a fifth of half a step."""
    k = 16_384
    a, b = _positive(1, k, 2000), _positive(2, k, 2000)
    want = a[:, ::15].double().t() @ b[:, ::15].double()
    off = ra.ra_linear_wgrad(a, b)[::15, ::15].double() / want - 1
    assert abs(float(off.mean())) < 2.0 ** -9 / 5 + MEAN


# (rows, k, cols) by how blocks share them: few rows, a tile's, two and four pairs, single blocks of 64 and 128 columns, pairs of
# 128 and 256, last tiles in parts
KINDS = [(16, 17_000, 500), (120, 16_392, 1000), (257, 16_400, 2081), (300, 16_392, 328), (256, 16_385, 4864), (520, 16_392, 3700),
         (512, 16_400, 3700), (2000, 16_392, 2000), (2500, 16_400, 2200)]


@pytest.mark.parametrize("m,k,n", KINDS)
def test_long_sums_in_bf16_of_every_kind(m, k, n):
    x, w, bias, residual = _normal(1, m, k), _normal(2, k, n, s=k ** -0.5), _normal(3, n, dtype=F32), _normal(4, m, n)
    kept = ra.Checkpoint8(m, n)
    got = ra.ra_linear(x, w, bias=bias, act="gelu", residual=residual, save=kept)
    z, size = x.double() @ w.double(), x.double().abs() @ w.double().abs()
    zb = z + bias.double()
    y = act64(zb, "gelu") + residual.double()
    off = sum_bound(k + 1) * (size + bias.double().abs())
    check(got, y, 1.13 * off + 2.0 ** -20 * zb.abs() + rounding(BF16) * y.abs() + 2.0 ** -20 * residual.double().abs())
    groups = -(-n // 32)
    top = torch.nn.functional.pad(zb.abs() + off, (0, groups * 32 - n)).view(m, groups, 32).amax(2).repeat_interleave(32, 1)[:, :n]
    check(ra.ra_checkpoint8_unpack(kept, dtype=F32), zb, top / 127.5 * (1 + 2.0 ** -20) + off)
    assert torch.equal(got, ra.ra_linear(x, w, bias=bias, act="gelu", residual=residual))
    wt, xt = w.t().contiguous(), x.t().contiguous()
    z8 = ra.ra_checkpoint8_pack(_normal(6, m, n, s=2.0))
    zz = values64(z8.q, z8.e, n)
    want = z * slope64(zz, "silu")
    check(ra.ra_linear_dgrad(x, wt, saved=z8, act="silu"), want,
          1.13 * sum_bound(k) * size + 2.0 ** -20 * z.abs() * (1 + zz.abs()) + rounding(BF16) * want.abs())
    held = _normal(7, m, n)
    want = z + held.double()
    dw, db = ra.ra_linear_wgrad(xt, w, bias_grad=True)
    check(dw, z, sum_bound(k) * size + rounding(BF16) * z.abs())
    check(db, w.double().sum(0), sum_bound(k) * w.double().abs().sum(0))
    ra.ra_linear_wgrad(xt, w, out=held, accumulate=True)
    check(held, want, sum_bound(k + 1) * (size + held.double().abs() + z.abs()) + rounding(BF16) * want.abs())
