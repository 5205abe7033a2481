"""Data-parallel training of a small model with this library alone: the
operators compute every worker's gradients, the ring averages them and takes
the SGD step.

    python -m examples.train_ffn [--workers 4] [--tokens 512] [--steps 30]

The model is one block of the Transformer whose gradients the library's
workloads average ("How GPipe works", section 1), without its attention: an
embedding V x d, scaled by sqrt(d), and a feed-forward layer d x h, h x d with
biases, GELU between them and the residual around them.  It learns the outputs
of a second such model with other weights (mean squared error).

Every logical worker has its own tokens and its own flat gradient row; all rows
lie in one GPU's memory.  A worker's step:

    forward   e  = ra_embedding_lookup(E, ids, sqrt(d))
              e8 = ra_checkpoint8_pack(e)                       kept for dW1
              a  = ra_linear(e, W1, b1, "gelu", save=z8)        z kept in 8 bits
              y  = ra_linear(a, W2, b2, residual=e)
    backward  dy                                                of the loss
              dW2, db2 = ra_linear_wgrad(z8, dy, "gelu")        a = gelu(z8), recomputed
              dz       = ra_linear_dgrad(dy, W2, z8, "gelu")
              dW1, db1 = ra_linear_wgrad(e8, dz)
              de       = ra_linear_dgrad(dz, W1, residual=dy)
              dE       = ra_embedding_grad(de, ids, V, sqrt(d))

The gradients are written straight into views of the worker's row.  Then
ra_allreduce_sgd leaves the mean of all rows in every row and w - lr * mean in
the binary32 weights, from which the next step's bf16 weights are taken.
"""
from __future__ import annotations

import argparse
from math import prod

import torch

import gradient_ring_all_gb300 as ra


def shapes(vocab: int, d: int, h: int):
    """The tensors in forward order, as they lie in the flat arrays."""
    return [("E", (vocab, d)), ("W1", (d, h)), ("b1", (h,)), ("W2", (h, d)), ("b2", (d,))]


def views(flat, layout):
    """The named tensors of a flat array."""
    out, at = {}, 0
    for name, shape in layout:
        out[name] = flat[at:at + prod(shape)].view(shape)
        at += prod(shape)
    return out


def initial(layout, generator):
    """Binary32 weights: normal, by fan-in; biases zero."""
    flat = torch.zeros(sum(prod(s) for _, s in layout), device="cuda")
    for name, t in views(flat, layout).items():
        if t.dim() == 2:
            t.normal_(0, t.shape[1 if name == "E" else 0] ** -0.5, generator=generator)
    return flat


class Model:
    """The weights as the operators take them: matrices in bf16, biases in binary32."""

    def __init__(self, flat, layout):
        v = views(flat, layout)
        self.E, self.W1, self.W2 = (v[n].bfloat16() for n in ("E", "W1", "W2"))
        self.b1, self.b2 = v["b1"], v["b2"]
        self.vocab, self.d = self.E.shape
        self.scale = self.d ** 0.5

    def forward(self, ids):
        """(y, what the backward pass needs)"""
        e = ra.ra_embedding_lookup(self.E, ids, scale=self.scale)
        z8 = ra.Checkpoint8(ids.numel(), self.W1.shape[1])
        a = ra.ra_linear(e, self.W1, bias=self.b1, act="gelu", save=z8)
        y = ra.ra_linear(a, self.W2, bias=self.b2, residual=e, dtype=torch.float32)
        return y, (ids, ra.ra_checkpoint8_pack(e), z8)

    def backward(self, dy, kept, grads):
        """Writes the gradients into `grads` (views of a worker's row)."""
        ids, e8, z8 = kept
        ra.ra_linear_wgrad(z8, dy, act="gelu", out=grads["W2"], bias_grad=grads["b2"])
        dz = ra.ra_linear_dgrad(dy, self.W2, saved=z8, act="gelu")
        ra.ra_linear_wgrad(e8, dz, out=grads["W1"], bias_grad=grads["b1"])
        de = ra.ra_linear_dgrad(dz, self.W1, residual=dy)
        ra.ra_embedding_grad(de, ids, self.vocab, scale=self.scale, out=grads["E"])


def gradients(model, teacher, ids, row, layout):
    """One worker's forward and backward pass; the loss as a device scalar."""
    y, kept = model.forward(ids)
    wanted, _ = teacher.forward(ids)
    off = y - wanted
    model.backward((off * (2.0 / off.numel())).bfloat16(), kept, views(row, layout))
    return off.square().mean()


def train(workers=4, tokens=512, steps=30, vocab=1000, d=256, h=1024, lr=2.0, seed=0):
    """The mean loss of each step."""
    layout = shapes(vocab, d, h)
    g = torch.Generator(device="cuda").manual_seed(seed)
    teacher = Model(initial(layout, g), layout)
    weights = initial(layout, g)
    views(weights, layout)["E"].copy_(teacher.E)  # the embedding starts near the teacher's, the layers do not
    rows = [torch.empty_like(weights) for _ in range(workers)]
    losses = []
    for _ in range(steps):
        model = Model(weights, layout)
        step = [gradients(model, teacher, torch.randint(0, vocab, (tokens,), generator=g, device="cuda"), row, layout) for row in rows]
        ra.ra_allreduce_sgd(rows, weights, lr)
        losses.append(torch.stack(step).mean())
    return torch.stack(losses).tolist()


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--workers", type=int, default=4)
    p.add_argument("--tokens", type=int, default=512, help="tokens a worker and step")
    p.add_argument("--steps", type=int, default=30)
    a = p.parse_args()
    losses = train(a.workers, a.tokens, a.steps)
    for k in range(0, len(losses), max(1, len(losses) // 10)):
        print("step %4d  loss %.5f" % (k, losses[k]))
    print("step %4d  loss %.5f" % (len(losses) - 1, losses[-1]))


if __name__ == "__main__":
    main()
