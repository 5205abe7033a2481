"""ra_logprobs on rows with finite masks, wide spreads and logits far from zero,
against the plain form in 64 bits and with the bounds of test_gpu_logprobs.py."""
from __future__ import annotations

import pytest
import torch

import gradient_ring_all_gb300 as ra
from test_gpu_logprobs import _check, _ids, _logits

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from gradient_ring_all_gb300 import build
    build.build()
    ra.load()


def _banned(vocab, share, seed):
    """A row's banned tokens: the first half, all but a share at random, or all."""
    if share == "half":
        return torch.arange(vocab, device="cuda") < vocab // 2
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.rand(vocab, generator=g, device="cuda") < share


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("vocab", [300, 513, 1024, 1500, 2048, 4001])
def test_many_alternatives_beside_the_lowest_value(vocab, dtype):
    """21 to 32 alternatives of rows in which the type's lowest value stands for banned tokens: each lane's logits count once."""
    z = _logits(12, vocab, dtype, seed=11).t.clone()
    for r in range(12):
        z[r, _banned(vocab, ("half", 0.5, 0.8, 0.95)[r % 4], r)] = torch.finfo(dtype).min
    ids = torch.full((12,), -1, device="cuda")
    for top in (20, 21, 27, 32):
        _check(z, ids, 1.0, top)


# a row of one warp, two, four, eight, several tiles, and a cluster's
VOCABS = [40, 1024, 1500, 6007, 12001, 32000, 70000, 131071]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("vocab", VOCABS)
@pytest.mark.parametrize("mask", [-1e4, -1e8, -1e9, -1e10, -1e20, "lowest"])
def test_finite_masks(mask, vocab, dtype):
    """Banned tokens at a finite value: the first half of a row, at random all but 5 %, and the whole row."""
    value = torch.finfo(dtype).min if mask == "lowest" else mask
    shares = ("half", 0.95, 1.0, 0.0)
    z = _logits(len(shares), vocab, dtype, seed=5).t.clone()
    for r, share in enumerate(shares):
        z[r, _banned(vocab, share, vocab)] = value
    ids = z.argmax(1)
    ids[3] = vocab  # padding
    for scale, top in ((1.0, 0), (1.0, 8), (0.8, 20), (0.8, 0), (1.0, 32)) + (() if mask == "lowest" else ((1.25, 0), (1.25, 8), (1.25, 32))):
        _check(z, ids, scale, top)
    if mask != "lowest":
        _check(z, torch.full_like(ids, vocab // 3), 1.0, 0)  # banned, in two rows or three


@pytest.mark.parametrize("vocab", [40, 40000])
def test_the_lowest_value_times_a_scale_above_one(vocab):
    """1.25 times the lowest value is no binary32 number: lse is minus infinity, the rest of the row as it should be."""
    for dtype in (F32, BF16):
        z = torch.full((1, vocab), torch.finfo(dtype).min, dtype=dtype, device="cuda")
        r = ra.ra_logprobs(z, torch.tensor([vocab - 1], device="cuda"), scale=1.25, entropy=True, top=3)
        even = torch.tensor(float(vocab), dtype=torch.float64).log().item()
        assert float(r.lse[0]) == -float("inf") and r.top_ids[0].tolist() == [0, 1, 2]
        for t in (-r.logp, r.entropy, -r.top_logp[0]):
            assert float((t.double() - even).abs().max()) < 1e-3


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("vocab", VOCABS)
def test_logits_far_from_zero(vocab, dtype):
    """Rows moved by up to 1e30, even ones among them, and scales that carry them there."""
    far = (1e5, -1e6, 1e6, -1e7, 1e7, 3e8, -1e9, 1e9, 1e30, -1e30)
    rows = [_logits(1, vocab, dtype, seed=k).t[0].float() + v for k, v in enumerate(far)] + [torch.full((vocab,), v, device="cuda") for v in far]
    z = torch.stack(rows).to(dtype)
    for scale, top in ((1.0, 0), (0.8, 8), (1.25, 0)):
        _check(z, _ids(len(rows), vocab), scale, top)
    z = _logits(4, vocab, dtype, seed=6).t
    for scale in (1e3, 1e5, 1e8, 1e30):
        _check(z, _ids(4, vocab), scale, 3)


def _first_batch(vocab, dtype):
    """As many logits as the threads of a row start from, and the few before them."""
    each = 8 if dtype == BF16 else 4
    vecs = -(-vocab // each)
    warps = 1 if vecs <= 512 else 2 if vecs <= 1024 else 4 if vecs <= 2048 else 8
    return warps * 32 * each * (2 if warps == 1 else 4) + each


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("vocab", [800, 1536, 6007, 12001, 20011, 70000, 131071])
def test_spreads(vocab, dtype):
    """A row's first logits, its last ones, or those of some lanes are far below the others, by gaps about which the sums
    leave binary32: the exponential's least argument, its flushed results, the sums' range."""
    gaps = (10.0, 20.0, 40.0, 60.0, 70.0, 81.0, 83.0, 84.0, 84.5, 85.0, 85.5, 87.0, 88.5, 90.0, 100.0, 110.0, 115.0, 120.0, 130.0, 150.0)
    first = min(_first_batch(vocab, dtype), vocab // 2)
    n = torch.arange(vocab, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(vocab)
    rows = []
    for gap in gaps:
        plain = torch.randn(vocab, generator=g, device="cuda")
        rows.append(torch.where(n < first, -gap, plain))
        for high in (4.0, 7.0):  # of one token among the first
            rows.append(torch.where(n == first // 3, high, rows[-1] if high == 4.0 else rows[-2]))
        rows.append(torch.where(n >= vocab - first, plain - gap, plain))
        rows.append(torch.where(n // 8 % 32 < 20, plain - gap, plain))
        rows.append(torch.where(n % (first + 77) == 5, plain, plain - gap))  # the high ones are few
    z = torch.stack(rows).to(dtype)
    ids = _ids(len(rows), vocab)
    for scale, top in ((1.0, 0), (1.0, 8), (0.8, 32)):
        _check(z, ids, scale, top)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("vocab", [1536, 12001, 40000])
def test_logits_that_rise_along_the_row(vocab, dtype):
    """Every batch is above the last one, from a little to so far that nothing is left of it."""
    n = torch.arange(vocab, device="cuda").double() / vocab
    z = torch.stack([n * rise for rise in (30.0, 300.0, 3e3, 3e4, 3e6, 1e12)] + [10.0 ** (n * 38), -(10.0 ** (38 - n * 38))]).to(dtype)
    for scale, top in ((1.0, 0), (1.0, 8), (0.7, 32)):
        _check(z, _ids(len(z), vocab), scale, top)
