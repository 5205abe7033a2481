"""ra_logprobs on rows with finite masks, against the plain form in 64 bits and with
the bounds of test_gpu_logprobs.py."""

import pytest
import torch

import gradient_ring_all_gb300 as ra
from test_gpu_logprobs import _check, _logits

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
