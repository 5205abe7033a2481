"""ra_logprobs_grad on rows with finite masks and rows whose lse is far from zero."""
from __future__ import annotations

import pytest
import torch

import gradient_ring_all_gb300 as ra
from block_reference import U, distribution64
from operator_reference import check
from test_gpu_logprobs import _check_grad, _ids, _logits

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from gradient_ring_all_gb300 import build
    build.build()
    ra.load()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("vocab", [40, 300, 1500, 40000])
@pytest.mark.parametrize("mask", [-1e4, -1e9, -1e20, "lowest"])
def test_finite_masks(mask, vocab, dtype):
    """Banned tokens get exactly 0 where p is 0 in binary32, the others their gradient."""
    value = torch.finfo(dtype).min if mask == "lowest" else mask
    z = _logits(3, vocab, dtype, seed=5).t.clone()
    n = torch.arange(vocab, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(vocab)
    z[0, n < vocab // 2] = value
    z[1, torch.rand(vocab, generator=g, device="cuda") < 0.9] = value
    z[2, n > 0] = value
    banned = z.float() <= -9000
    ids = z.argmax(1)
    ids[1] = int(banned[1].int().argmax())  # a banned one
    for scale, entropy in ((1.0, False), (0.8, True)):
        got = _check_grad(z, ids, scale, entropy)
        banned[1, ids[1]] = False
        assert not bool(got[banned].any())


@pytest.mark.parametrize("scale", [0.7, 1.0, 1.3])
@pytest.mark.parametrize("vocab", [300, 3000])
def test_p_keeps_what_lse_leaves(vocab, scale):
    """p is off by 2^-24 |lse| of itself and no more, beside what rows near zero lose: lse's sum (as there), one rounding of its
    argument and of the product with log2 e, the exponential's 2^-21, three factors of the gradient."""
    rows = 64
    z = _logits(rows, vocab, F32, seed=8).t + torch.linspace(-2.0 ** 17, 2.0 ** 17, rows, device="cuda").unsqueeze(1)
    ids = torch.full((rows,), -1, device="cuda")
    ids[::2] = torch.arange(0, rows, 2, device="cuda")
    r = ra.ra_logprobs(z, ids, scale=scale)
    s = float(torch.tensor(scale, dtype=F32))
    y, m, log_s, h, p = distribution64(z, s)
    lse = m + log_s
    g = torch.linspace(-2, 2, rows, device="cuda")
    got = ra.ra_logprobs_grad(z, ids, r.lse, g, scale=scale)
    gd = torch.where(ids >= 0, g, 0.0).double().unsqueeze(1)
    want = -gd * p
    inside = torch.arange(0, rows, 2, device="cuda")
    want[inside, ids[inside]] += gd[inside, 0]
    d = (y - lse.unsqueeze(1)).abs()
    rel = U * lse.abs() + (408 + 8 * (log_s + h)) * U
    rel = torch.expm1(rel.unsqueeze(1) + 4 * U * d + 2.0 ** -21)
    check(got, want * s, s * (rel * gd.abs() * p + 4 * U * (gd.abs() * p + want.abs())) + 2.0 ** -126, "gradient")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("vocab", [40, 300, 1500, 40000])
def test_rows_of_which_lse_says_nothing(vocab, dtype):
    """Rows masked throughout by a finite value whose lse is below -2^24 have no gradient; above 2^24 p stays below 1."""
    low = [torch.full((vocab,), v, device="cuda") for v in (-3e7, -1e8, -1e9, -1.1e9, -1e10, -1e20, torch.finfo(dtype).min)]
    z = torch.stack(low + [_logits(1, vocab, F32, seed=3).t[0] - 1e9]).to(dtype)
    ids = _ids(len(z), vocab)
    for scale in (1.0, 0.8, 1.25, 0.7):
        r = ra.ra_logprobs(z, ids, scale=scale, entropy=True)
        g = torch.full((len(z),), 3.0, device="cuda")
        for got in (ra.ra_logprobs_grad(z, ids, r.lse, g, scale=scale), ra.ra_logprobs_grad(z, ids, r.lse, g, scale=scale, entropy=r.entropy, grad_entropy=g)):
            assert not bool(got.any())
    z = torch.stack([torch.full((vocab,), v, device="cuda") + torch.randn(vocab, device="cuda") for v in (3e7, 1e9, 1.1e9, 1e10, 1e20, 1e30)]).to(dtype)
    for scale in (1.0, 0.8, 1.25, 0.7):
        ids = torch.zeros(len(z), dtype=torch.int64, device="cuda")
        r = ra.ra_logprobs(z, ids, scale=scale)
        got = ra.ra_logprobs_grad(z, ids, r.lse, torch.full((len(z),), 3.0, device="cuda"), scale=scale).float()
        assert float(got.abs().max()) <= 3.0 * scale * 1.01
