"""ra_logprobs on rows with finite masks and logits far from zero, against the plain
form in 64 bits and with the bounds of test_gpu_logprobs.py."""
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
