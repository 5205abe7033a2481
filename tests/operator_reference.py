"""Plain references of the training-step operators in 64 bits, and the error
bounds the tests hold the kernels to.

The bounds.  u = 2^-24 is binary32's unit roundoff.  A sum of k products of
bf16 values (each product exact in binary32), added in any order and any
grouping by additions that round to nearest or truncate, is off by at most
2 k u times the sum of the products' magnitudes (first order; each of at most
k additions is off by 2u of a partial sum that those magnitudes bound).  An
activation's slope is at most 1.13, so it carries an error on at most 1.13
times as large; its own evaluation is allowed 2^-20 of |z| (erf and exp of the
CUDA library are within a few units in the last place, their arguments are
rounded once, and |z| bounds the result and the size of z times the slope's
change).  The result's rounding adds 2^-9 (bf16) or 2^-24 (binary32) of its
magnitude, doubled where a residual is added before it."""
from __future__ import annotations

import math

import torch

U = 2.0 ** -24
GROUP = 32


def sum_bound(terms: int) -> float:
    return 2 * (terms + 4) * U


def rounding(dtype) -> float:
    return 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -23


def act64(z, act):
    if act == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if act == "gelu":
        return z * 0.5 * torch.special.erfc(-z / math.sqrt(2))
    if act == "silu":
        return z * torch.sigmoid(z)
    return z


def slope64(z, act):
    if act == "relu":
        return (z > 0).double()
    if act == "gelu":
        return 0.5 * torch.special.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == "silu":
        p = torch.sigmoid(z)
        return p + z * p * (1 - p)
    return torch.ones_like(z)


def power64(n):
    """2^n in 64 bits from the exponent's bits (torch.ldexp takes a power in binary32), |n| < 1000."""
    return ((n.to(torch.int64) + 1023) << 52).view(torch.float64)


def pack64(x):
    """(q, e) of a finite matrix by the definition: frexp for the exponent, whole steps in 64 bits."""
    rows, cols = x.shape
    groups = -(-cols // GROUP)
    full = torch.zeros(rows, groups * GROUP, dtype=torch.float64, device=x.device)
    full[:, :cols] = x.double()
    full = full.view(rows, groups, GROUP)
    top = full.abs().amax(2) if cols else full.new_zeros(rows, 0)
    half, power = torch.frexp(top)
    power = power.to(torch.int64) - 1 + (2 * half >= 255 / 128)
    e = torch.where(top > 0, (power - 6 + 127).clamp(1, 248), torch.ones_like(power))
    full = torch.where((top >= 255 * 2.0 ** 120).unsqueeze(2), full * (127 / 128), full)  # the top of binary32
    q = torch.round(full * power64(127 - e).unsqueeze(2))
    return q.to(torch.int8).view(rows, -1), e.to(torch.uint8)


def values64(q, e, cols):
    rows, groups = e.shape
    v = q.double().view(rows, groups, GROUP) * power64(e.to(torch.int64) - 127).unsqueeze(2)
    return v.view(rows, -1)[:, :cols]


def check(got, want, bound, what=""):
    """|got - want| <= bound everywhere; non-finite values of `want` are met as they are."""
    got = got.double()
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), "%s: NaN elsewhere than expected" % what
    odd = ~fine & ~torch.isnan(want)
    assert torch.equal(got[odd], want[odd]), "%s: another infinity than expected" % what
    off = (got - want).abs()[fine] - torch.broadcast_to(torch.as_tensor(bound, dtype=torch.float64, device=want.device), want.shape)[fine]
    assert off.numel() == 0 or off.max().item() <= 0, "%s: %d of %d values are off, the worst by %.3g over its bound" % (
        what, int((off > 0).sum()), off.numel(), off.max().item())


class Framed:
    """A rows x cols matrix inside a larger one filled with a pattern: `lead` elements before each row's start, `gap` after
    its end, so writes outside it show."""

    def __init__(self, rows, cols, dtype, lead=0, gap=0):
        self.rows, self.cols, self.lead = rows, cols, lead
        self.base = torch.empty(rows + 2, lead + cols + gap, dtype=dtype, device="cuda")
        self.raw = self.base.view(torch.int16 if dtype == torch.bfloat16 else torch.int32 if dtype == torch.float32 else torch.int8)
        self.raw.fill_(0x5A)
        self.t = self.base[1:rows + 1, lead:lead + cols]

    def fill(self, src):
        self.t.copy_(src)
        return self

    def intact(self, what=""):
        seen = self.raw.clone()
        seen[1:self.rows + 1, self.lead:self.lead + self.cols] = 0x5A
        assert bool((seen == 0x5A).all()), "%s: something outside the matrix was written" % what
