"""examples/train_ffn.py: the operators, the ring and the SGD step together."""
from __future__ import annotations

import pytest
import torch

import gradient_ring_all_gb300 as ra
from operator_reference import act64, slope64, values64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from gradient_ring_all_gb300 import build
    build.build()
    ra.load()


def test_it_learns_and_repeats():
    from examples import train_ffn
    losses = train_ffn.train(workers=3, tokens=200, steps=25)
    assert losses[-1] < 0.5 * losses[0]
    assert losses == train_ffn.train(workers=3, tokens=200, steps=25)  # every sum has a fixed order


def test_workers_gradients_average_to_the_whole_batch():
    """Four workers' averaged gradients against the gradient of all their
    tokens at once, computed in 64 bits from the same bf16 weights and the
    same 8-bit checkpoints (data parallelism with equal shards)."""
    from examples import train_ffn
    vocab, d, h, n, tokens = 50, 64, 96, 4, 130
    layout = train_ffn.shapes(vocab, d, h)
    g = torch.Generator(device="cuda").manual_seed(3)
    model = train_ffn.Model(train_ffn.initial(layout, g), layout)
    ids = [torch.randint(0, vocab, (tokens,), generator=g, device="cuda") for _ in range(n)]
    dy = [(torch.randn(tokens, d, generator=g, device="cuda") * 1e-2).bfloat16() for _ in range(n)]
    size = sum(t.numel() for t in (model.E, model.W1, model.b1, model.W2, model.b2))
    rows = [torch.empty(size, device="cuda") for _ in range(n)]
    want = {name: 0 for name, _ in layout}
    for k in range(n):
        _, kept = model.forward(ids[k])
        model.backward(dy[k], kept, train_ffn.views(rows[k], layout))
        _, e8, z8 = kept
        e, z, dy64 = values64(e8.q, e8.e, d), values64(z8.q, z8.e, h), dy[k].double()
        dz = (dy64 @ model.W2.double().t()) * slope64(z, "gelu")
        de = dz @ model.W1.double().t() + dy64
        table = torch.zeros(vocab, d, dtype=torch.float64, device="cuda").index_add_(0, ids[k], de) * model.scale
        for name, t in (("E", table), ("W1", e.t() @ dz), ("b1", dz.sum(0)), ("W2", act64(z, "gelu").t() @ dy64), ("b2", dy64.sum(0))):
            want[name] = want[name] + t / n
    ra.ra_allreduce_avg(rows)
    got = train_ffn.views(rows[0], layout)
    for name, t in want.items():
        # bf16 roundings of dz, de and gelu(z): a few times 2^-9 of the tensor's size
        off = float((got[name].double() - t).norm() / t.norm())
        assert off < 4 * 2.0 ** -9, (name, off)
