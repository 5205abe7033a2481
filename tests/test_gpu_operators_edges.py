"""Edges of the operators: empty checkpoints, sums with no rows, a bias
gradient alone."""
from __future__ import annotations

import pytest
import torch

import gradient_ring_all_gb300 as ra
from operator_reference import check, sum_bound

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
ACTS = ["none", "relu", "gelu", "silu"]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from gradient_ring_all_gb300 import build
    build.build()
    ra.load()


def _normal(seed, *shape, dtype=BF16, s=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * s).to(dtype)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("out_type", [BF16, F32])
def test_weight_gradient_of_no_tokens(act, out_type):
    """No rows: zero sums, and accumulated ones stay."""
    k, n = 24, 40
    kept, dy = ra.Checkpoint8(0, k), torch.empty(0, n, dtype=BF16, device="cuda")
    dw, db = ra.ra_linear_wgrad(kept, dy, act=act, dtype=out_type, bias_grad=True)
    assert dw.shape == (k, n) and not bool(dw.any()) and db.shape == (n,) and not bool(db.any())
    held, hb = torch.full((k, n), 2.0, dtype=out_type, device="cuda"), torch.full((n,), 3.0, device="cuda")
    ra.ra_linear_wgrad(kept, dy, act=act, out=held, bias_grad=hb, accumulate=True)
    assert bool((held == 2).all()) and bool((hb == 3).all())


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m", [1, 100, 512, 513, 3000])
@pytest.mark.parametrize("n", [40, 67])
def test_bias_gradient_alone(act, m, n):
    """An input without columns leaves the column sums of dy, on both sides of the number of rows at which they get a launch
    of their own; accumulated they add."""
    dy = _normal(m, m, n)
    want, bound = dy.double().sum(0), sum_bound(m) * dy.double().abs().sum(0)
    kept = ra.Checkpoint8(m, 0)
    dw, db = ra.ra_linear_wgrad(kept, dy, act=act, bias_grad=True)
    assert dw.shape == (0, n)
    check(db, want, bound)
    ra.ra_linear_wgrad(kept, dy, act=act, out=dw, bias_grad=db, accumulate=True)
    check(db, 2 * want, 2 * bound + 2.0 ** -23 * want.abs())
    if act == "none":
        _, again = ra.ra_linear_wgrad(torch.empty(m, 0, dtype=BF16, device="cuda"), dy, bias_grad=True)
        check(again, want, bound)


@pytest.mark.parametrize("out_type", [BF16, F32])
@pytest.mark.parametrize("k", [64, 600])
def test_one_row_in_place_whatever_its_stride(k, out_type):
    """A single row has no stride: the residual may be the output under another one."""
    n = 96
    x, w, r = _normal(1, 1, k), _normal(2, k, n, s=k ** -0.5), _normal(3, 1, n, dtype=out_type)
    want = ra.ra_linear(x, w, residual=r, dtype=out_type)
    for lda, ldb in ((n, n + 32), (n + 7, n), (1, n)):
        both = torch.cat([r.flatten(), torch.zeros(64, dtype=out_type, device="cuda")])
        ra.ra_linear(x, w, residual=both.as_strided((1, n), (lda, 1)), out=both.as_strided((1, n), (ldb, 1)))
        assert torch.equal(both[:n], want[0]) and not bool(both[n:].any())
        both[:n] = r[0]
        ra.ra_linear_dgrad(x, w.t().contiguous(), residual=both.as_strided((1, n), (lda, 1)), out=both.as_strided((1, n), (ldb, 1)))
        check(both[None, :n], x.double() @ w.double() + r.double(), sum_bound(k) * (x.double().abs() @ w.double().abs()) + 2.0 ** -7 * (
            (x.double() @ w.double()).abs() + r.double().abs()))
    with pytest.raises(ra.RaError, match="OVERLAP"):  # a part of the row in place is not
        both = torch.zeros(2 * n, dtype=out_type, device="cuda")
        ra.ra_linear(x, w, residual=both[8:8 + n].view(1, n), out=both[:n].view(1, n))


@pytest.mark.parametrize("d", [2_097_120, 2_097_121, (1 << 22) + 5, (1 << 23) + 1024])
@pytest.mark.parametrize("out_type", [BF16, F32])
def test_table_gradient_of_very_wide_rows(d, out_type):
    """Any width below 2^31: the columns go out in as many launches as they need, the runs that cross pieces are listed once.
    The sums are exact (small whole numbers)."""
    tokens, vocab = 27, 3
    ids = torch.tensor([0, 2, -1, 2], device="cuda").repeat(7)[:tokens]
    grad = torch.randint(-3, 4, (tokens, d), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda", dtype=torch.int8).to(BF16)
    want = torch.zeros(vocab, d, device="cuda").index_add_(0, ids[ids >= 0], grad[ids >= 0].float())
    got = ra.ra_embedding_grad(grad, ids, vocab, dtype=out_type)
    assert torch.equal(got.float(), want)
    ra.ra_embedding_grad(grad, ids, vocab, out=got, accumulate=True)
    assert torch.equal(got.float(), 2 * want)
    assert torch.equal(ra.ra_embedding_lookup(got, ids[:1]).float(), 2 * want[:1])


@pytest.mark.parametrize("top_steps", [100.0, 127.25, 127.5, 127.75, 127.99999])
@pytest.mark.parametrize("power", [-126, -120, 0, 100, 120, 121])
def test_checkpoint_error_by_magnitude(top_steps, power):
    """Off by at most half a step, also where the step is held at 2^-126; at the very top of binary32, where a group is taken
    times 127/128, by 1.5 steps (the scaling's 128 / 128 and the rounding's half)."""
    g = torch.Generator(device="cuda").manual_seed(1)
    x = (torch.rand(64, 32, generator=g, device="cuda", dtype=torch.float64) * 2 - 1) * top_steps
    x[:, 3] = top_steps
    x[::2, 7] = -top_steps + 0.25
    x = (x * 2.0 ** power).float()
    assert bool(torch.isfinite(x).all())
    kept = ra.ra_checkpoint8_pack(x)
    back = ra.ra_checkpoint8_unpack(kept, dtype=F32).double()
    assert bool(torch.isfinite(back).all())
    step = torch.exp2(kept.e.double() - 127).repeat_interleave(32, 1)
    scaled = x.abs().amax(1, keepdim=True).double() >= 255 * 2.0 ** 120
    limit = torch.where(scaled, 1.5, 0.5) * step
    off = (back - x.double()).abs()
    assert bool((off <= limit).all())
    assert bool(scaled.any()) == (power == 121 and top_steps >= 127.5)
    top = x.abs().amax(1, keepdim=True).double()
    assert bool((off <= torch.where(scaled, top / 85, torch.clamp(top / 127.5, min=2.0 ** -127))).all())
