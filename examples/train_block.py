"""Data-parallel training of a small language model with this library alone: the
operators compute every worker's loss and gradients, the ring averages them and
takes the SGD step.

    python -m examples.train_block [--workers 4] [--tokens 512] [--steps 40]

The model is the feed-forward half of a Transformer block between an embedding and
a softmax projection ("How GPipe works", section 1: V x d embedding and projection,
d x h and h x d weights with biases, layer norms with gain and bias), with a norm
behind the block as well as before it, a learned gate and dropout.  It learns the
next token of a random walk in which every token has a few likely followers.

Every logical worker has its own tokens and its own flat gradient row.  A worker's
step:

    forward   x0           = ra_embedding_lookup(E, ids, sqrt(d))
              h1, k1       = ra_norm_block(x0, pre=N1)
              a            = ra_linear(h1, W1, b1, "gelu", save=z8)       z kept in 8 bits
              f            = ra_dropout(ra_linear(a, W2, b2), p, seed)    no mask is kept
              x1, h2, k2   = ra_norm_block(x0, f, post=Np, gate=g, pre=N2)
              logits       = ra_linear(h2, U)
              logp, lse    = ra_logprobs(logits, next)
    backward  dlogits      = ra_logprobs_grad(logits, next, lse, -1/n)    in the logits' place
              dU, dh2      = ra_linear_wgrad, ra_linear_dgrad
              dx, df, ...  = ra_norm_block_grad(dh2, x1, k2, f, Np, g, N2)
              df           = ra_dropout(df, p, seed)                      the same mask again
              dW2, db2, dz, dW1, db1, dh1  as in train_ffn.py
              dx, ...      = ra_norm_block_grad(dh1, x0, k1, N1, dx)      added to the stream's
              dE           = ra_embedding_grad(dx, ids, V, sqrt(d))

The gradients are written straight into views of the worker's row.  The mask of a
worker is that of its rows of the whole batch (first_row), so the same batch spread
over another number of workers drops the same values.
"""
from __future__ import annotations

import argparse

import torch

import gradient_ring_all_gb300 as ra
from examples.train_ffn import views

SITE = 1  # of the model's one dropout


def shapes(vocab: int, d: int, h: int):
    """The tensors in forward order, as they lie in the flat arrays."""
    return [("E", (vocab, d)), ("g1", (d,)), ("c1", (d,)), ("W1", (d, h)), ("b1", (h,)), ("W2", (h, d)), ("b2", (d,)), ("gp", (d,)), ("cp", (d,)),
            ("gate", (d,)), ("g2", (d,)), ("c2", (d,)), ("U", (d, vocab))]


def initial(layout, generator):
    """Binary32 weights: matrices normal, by fan-in; gains and the gate one; biases zero."""
    flat = torch.zeros(sum(torch.Size(s).numel() for _, s in layout), device="cuda")
    for name, t in views(flat, layout).items():
        if t.dim() == 2:
            t.normal_(0, t.shape[1 if name == "E" else 0] ** -0.5, generator=generator)
        elif name in ("g1", "gp", "g2", "gate"):
            t.fill_(1.0)
    return flat


class Model:
    """The weights as the operators take them: matrices in bf16, vectors in binary32."""

    def __init__(self, flat, layout, p: float = 0.1):
        self.v = v = views(flat, layout)
        self.E, self.W1, self.W2, self.U = (v[n].bfloat16() for n in ("E", "W1", "W2", "U"))
        self.before, self.behind, self.last = ra.Norm(v["g1"], v["c1"]), ra.Norm(v["gp"], v["cp"]), ra.Norm(v["g2"], v["c2"])
        self.vocab, self.d = self.E.shape
        self.p, self.scale = p, self.d ** 0.5

    def forward(self, ids, targets, seed, first_row: int = 0):
        """(log probabilities of the targets, what the backward pass needs)"""
        x0 = ra.ra_embedding_lookup(self.E, ids, scale=self.scale)
        _, h1, k1 = ra.ra_norm_block(x0, pre=self.before)
        z8 = ra.Checkpoint8(ids.numel(), self.W1.shape[1])
        a = ra.ra_linear(h1, self.W1, bias=self.v["b1"], act="gelu", save=z8)
        f = ra.ra_linear(a, self.W2, bias=self.v["b2"])
        ra.ra_dropout(f, self.p, seed, site=SITE, first_row=first_row, out=f)
        x1, h2, k2 = ra.ra_norm_block(x0, f, post=self.behind, gate=self.v["gate"], pre=self.last)
        logits = ra.ra_linear(h2, self.U)
        r = ra.ra_logprobs(logits, targets)
        return r.logp, (ids, targets, seed, first_row, x0, h1, k1, z8, f, x1, h2, k2, logits, r.lse)

    def backward(self, g, kept, grads):
        """From the log probabilities' gradient g; writes into `grads` (views of a worker's row)."""
        ids, targets, seed, first_row, x0, h1, k1, z8, f, x1, h2, k2, logits, lse = kept
        dlogits = ra.ra_logprobs_grad(logits, targets, lse, g, out=logits)
        ra.ra_linear_wgrad(h2, dlogits, out=grads["U"])
        dh2 = ra.ra_linear_dgrad(dlogits, self.U)
        out = ra.NormBlockGrads(dx=torch.empty_like(x1), df=torch.empty_like(f), gate=grads["gate"], post_gain=grads["gp"], post_bias=grads["cp"],
                                pre_gain=grads["g2"], pre_bias=grads["c2"])
        ra.ra_norm_block_grad(dh2, x1, k2, f=f, post=self.behind, gate=self.v["gate"], pre=self.last, out=out)
        df = ra.ra_dropout(out.df, self.p, seed, site=SITE, first_row=first_row, out=out.df)
        ra.ra_linear_wgrad(z8, df, act="gelu", out=grads["W2"], bias_grad=grads["b2"])
        dz = ra.ra_linear_dgrad(df, self.W2, saved=z8, act="gelu")
        ra.ra_linear_wgrad(h1, dz, out=grads["W1"], bias_grad=grads["b1"])
        dh1 = ra.ra_linear_dgrad(dz, self.W1)
        ra.ra_norm_block_grad(dh1, x0, k1, pre=self.before, dx=out.dx, out=ra.NormBlockGrads(dx=out.dx, pre_gain=grads["g1"], pre_bias=grads["c1"]))
        ra.ra_embedding_grad(out.dx, ids, self.vocab, scale=self.scale, out=grads["E"])


def gradients(model, ids, targets, seed, first_row, row, layout):
    """One worker's forward and backward pass; the loss as a device scalar."""
    logp, kept = model.forward(ids, targets, seed, first_row)
    model.backward(torch.full_like(logp, -1.0 / logp.numel()), kept, views(row, layout))
    return -logp.mean()


def walk(followers, tokens, generator):
    """`tokens` tokens and their followers, each one of the few that the token has."""
    ids = torch.randint(0, followers.shape[0], (tokens,), generator=generator, device="cuda")
    which = torch.randint(0, followers.shape[1], (tokens,), generator=generator, device="cuda")
    return ids, followers[ids, which]


def train(workers=4, tokens=512, steps=40, vocab=500, d=128, h=512, lr=1.0, p=0.1, seed=0):
    """The mean loss of each step."""
    layout = shapes(vocab, d, h)
    g = torch.Generator(device="cuda").manual_seed(seed)
    followers = torch.randint(0, vocab, (vocab, 2), generator=g, device="cuda")
    weights = initial(layout, g)
    rows = [torch.empty_like(weights) for _ in range(workers)]
    losses = []
    for step in range(steps):
        model = Model(weights, layout, p)
        parts = []
        for k, row in enumerate(rows):
            ids, targets = walk(followers, tokens, g)
            parts.append(gradients(model, ids, targets, seed * 1_000_003 + step, k * tokens, row, layout))
        ra.ra_allreduce_sgd(rows, weights, lr)
        losses.append(torch.stack(parts).mean())
    return torch.stack(losses).tolist()


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--workers", type=int, default=4)
    p.add_argument("--tokens", type=int, default=512, help="tokens a worker and step")
    p.add_argument("--steps", type=int, default=40)
    a = p.parse_args()
    losses = train(a.workers, a.tokens, a.steps)
    for k in range(0, len(losses), max(1, len(losses) // 10)):
        print("step %4d  loss %.5f" % (k, losses[k]))
    print("step %4d  loss %.5f" % (len(losses) - 1, losses[-1]))


if __name__ == "__main__":
    main()
