"""The operators between a step's products together, as a training step uses them:
examples/train_block.py's gradients against 64 bits, and a captured step."""
from __future__ import annotations

import math

import pytest
import torch

import gradient_ring_all_gb300 as ra
from block_reference import keep_mask

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from gradient_ring_all_gb300 import build
    build.build()
    ra.load()


def _norm(v, gain, bias):
    c = v - v.mean(1, keepdim=True)
    return c * (c.square().mean(1, keepdim=True) + 1e-5).rsqrt() * gain + bias


def _loss64(w, ids, targets, keep, p):
    """The model in 64 bits by torch's own derivatives; w: the leaves."""
    x0 = w["E"][ids] * math.sqrt(w["E"].shape[1])
    z = _norm(x0, w["g1"], w["c1"]) @ w["W1"] + w["b1"]
    f = (0.5 * z * torch.special.erfc(-z / math.sqrt(2))) @ w["W2"] + w["b2"]
    t = round(65536 * p)
    f = torch.where(keep, f * (65536 / (65536 - t)), 0.0)
    x1 = x0 + w["gate"] * _norm(f, w["gp"], w["cp"])
    logits = _norm(x1, w["g2"], w["c2"]) @ w["U"]
    return -torch.log_softmax(logits, 1).gather(1, targets.unsqueeze(1)).mean()


def test_workers_gradients_average_to_the_whole_batch():
    """Three workers' averaged gradients against the derivatives, in 64 bits, of the loss of all their tokens at once: the same
    bf16 weights, the mask of the whole batch.

    The bound: every tensor that is handed on is rounded to bf16, by 2^-9 / sqrt 3 of a value in the mean square; a gradient has
    at most 16 such roundings before it, which are independent: 16^(1/2) 2^-9 / sqrt 3 = 0.5 %.  The pre-activation is kept in
    steps of 1/64 of its group's largest power of two, 1/32 of its deviation as a rule: 1/32 / sqrt 12 = 0.9 % of it, which the
    slope of gelu (its own slope is 0.8 at most) carries into dz.  Together 1.1 %; twice that is allowed."""
    from examples import train_block
    vocab, d, h, n, tokens, p, seed = 70, 64, 96, 3, 130, 0.2, 12345
    layout = train_block.shapes(vocab, d, h)
    g = torch.Generator(device="cuda").manual_seed(3)
    flat = train_block.initial(layout, g)
    for name, t in train_block.views(flat, layout).items():
        if t.dim() == 1:
            t.add_(torch.randn(t.shape, generator=g, device="cuda") * 0.1)
    model = train_block.Model(flat, layout, p)
    ids, targets = (torch.randint(0, vocab, (n * tokens,), generator=g, device="cuda") for _ in range(2))
    rows = [torch.full_like(flat, float("nan")) for _ in range(n)]
    losses = [train_block.gradients(model, ids[k * tokens:(k + 1) * tokens], targets[k * tokens:(k + 1) * tokens], seed, k * tokens, rows[k], layout)
              for k in range(n)]
    ra.ra_allreduce_avg(rows)
    leaves = {name: {"E": model.E, "W1": model.W1, "W2": model.W2, "U": model.U}.get(name, t).double().clone().requires_grad_()
              for name, t in train_block.views(flat, layout).items()}
    keep = keep_mask(n * tokens, d, p, seed, train_block.SITE).cuda()
    loss = _loss64(leaves, ids, targets, keep, p)
    loss.backward()
    # the logits are rounded to bf16 (2^-9 of values below 4), their mean over the tokens far less
    assert abs(float(torch.stack(losses).mean()) - float(loss.detach())) < 4 * 2.0 ** -9
    for name, got in train_block.views(rows[0], layout).items():
        want = leaves[name].grad
        off = float((got.double() - want).norm() / want.norm())
        assert off < 0.022, (name, off)


def test_it_runs_and_repeats():
    from examples import train_block
    losses = train_block.train(workers=2, tokens=100, steps=4)
    assert all(math.isfinite(v) for v in losses)
    assert losses == train_block.train(workers=2, tokens=100, steps=4)  # every sum has a fixed order


def test_another_number_of_workers_drops_the_same_values():
    """The batch whole and in micro-batches: the same mask, so the same log probabilities."""
    from examples import train_block
    layout = train_block.shapes(50, 64, 96)
    g = torch.Generator(device="cuda").manual_seed(5)
    model = train_block.Model(train_block.initial(layout, g), layout, 0.3)
    ids, targets = (torch.randint(0, 50, (96,), generator=g, device="cuda") for _ in range(2))
    whole, _ = model.forward(ids, targets, 9)
    parts = torch.cat([model.forward(ids[a:a + 32], targets[a:a + 32], 9, first_row=a)[0] for a in (0, 32, 64)])
    # the linear layer's products may be grouped by other tiles; bf16 steps of logits below 8
    assert float((whole - parts).abs().max()) < 8 * 2.0 ** -8
    other, _ = model.forward(ids[32:64], targets[32:64], 9)
    assert float((whole[32:64] - other).abs().max()) > 8 * 2.0 ** -8  # without first_row the mask is another


def test_a_captured_step_with_a_seed_in_device_memory():
    """Forward and backward in one graph, while an eager pass has used the same weights; every replay takes the next mask."""
    from examples import train_block
    layout = train_block.shapes(40, 64, 96)
    g = torch.Generator(device="cuda").manual_seed(6)
    flat = train_block.initial(layout, g)
    model = train_block.Model(flat, layout, 0.5)
    ids, targets = (torch.randint(0, 40, (60,), generator=g, device="cuda") for _ in range(2))
    row, eager = torch.empty_like(flat), torch.empty_like(flat)
    train_block.gradients(model, ids, targets, 7, 0, row, layout)
    seed = torch.tensor([7], dtype=torch.int64, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss = train_block.gradients(model, ids, targets, seed, 0, row, layout)
        seed.add_(1)
    for k in range(3):
        graph.replay()
        want = train_block.gradients(model, ids, targets, 7 + k, 0, eager, layout)
        assert torch.equal(row, eager) and torch.equal(loss, want)
