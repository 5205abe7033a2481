"""The operators between a training step's products, from the blocks to the
loss: what they compute, and the cases they are measured on.

- ``dropout``       residual + x * keep / (1 - p), the mask made from a seed and
                    the value's place alone, so that the backward pass (the same
                    call on the gradient) and a recomputation make it again
- ``norm_block``    the join behind one block and the norm before the next:
                    x' = a x + b gate * norm(f), h = norm(x')
- ``norm_grad``     its gradients: of the stream, the block's output, the gate,
                    both norms' gains and biases
- ``logprobs``      log probabilities of given tokens with their distribution's
                    entropy and its most likely alternatives
- ``logprobs_grad`` the logits' gradient from those of log probability and entropy

``run`` computes each in elementary torch operations in 32 bits, or, with
``own`` true, through the package's calls on the same inputs.  ``exact`` is the
definition in 64 bits.

The mask: Philox4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel random
numbers: as easy as 1, 2, 3", 2011) under the 64-bit seed as key gives 128 bits
for the counter (column / 8, site, row, row / 2^32); column 8 g + j has 16 of
them, the low half of word j / 2 for an even j and the high half for an odd
one.  A value is kept where these 16 bits are at least t = 65536 p, rounded to
a whole number, and then scaled by 65536 / (65536 - t).

A norm is (v - m) * rstd * gain + bias over a row, m its mean ("layer") or 0
("rms") and rstd = (mean (v - m)^2 + eps)^-1/2.  The stream x' is rounded to
its type before its norm is taken, as the backward pass reads it so.  Kept for
the backward pass: m and rstd of both norms, four numbers a row.

Sizes: the Transformer of the package's workloads (d 2048, ffn 8192, vocabulary
32000, 8192 tokens a step), a byte-level vocabulary, and odd ones.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32
TYPES = {"bf16": BF16, "f32": F32}
SIZE = {"bf16": 2, "f32": 4}
EPS = 1e-5
BANNED = -math.inf


def listed():
    return [
        # a sublayer's output on its way into the residual stream
        dict(name="dropout_sublayer", op="dropout", rows=8192, cols=2048, dtype="bf16", p=0.1, residual=True),
        # the ffn's hidden activation (and, the same call, its gradient)
        dict(name="dropout_hidden", op="dropout", rows=8192, cols=8192, dtype="bf16", p=0.1, residual=False),
        # a small odd micro-batch in binary32: rows share no 16-byte boundary
        dict(name="dropout_odd", op="dropout", rows=333, cols=1001, dtype="f32", p=0.5, residual=True),
        # behind a block and before the next one, for a step's tokens
        dict(name="norm_block_step", op="norm_block", rows=8192, d=2048, kind="layer", stream="bf16", block="bf16", join=True, gate="vector"),
        # the same for a single token: latency
        dict(name="norm_block_token", op="norm_block", rows=1, d=2048, kind="rms", stream="f32", block="bf16", join=True, gate="vector"),
        # the norm before a first block, on wide rows of a binary32 stream
        dict(name="norm_block_wide", op="norm_block", rows=2048, d=8192, kind="rms", stream="f32", block="bf16", join=False, gate="none"),
        # the backward pass of norm_block_step
        dict(name="norm_grad_step", op="norm_grad", rows=8192, d=2048, kind="layer", stream="bf16", block="bf16", join=True, gate="vector"),
        # a ragged micro-batch in binary32, every token with a gate of its own
        dict(name="norm_grad_ragged", op="norm_grad", rows=777, d=1003, kind="rms", stream="f32", block="f32", join=True, gate="matrix"),
        # the loss of a step's tokens with what a log of the run shows beside it; the batch ends in padding
        dict(name="logprobs_step", op="logprobs", rows=8192, vocab=32000, dtype="bf16", scale=1.0, top=8, pad=100, banned=0.0),
        # the next token of 16 answers: a long odd vocabulary, a temperature, tokens that are not allowed
        dict(name="logprobs_answers", op="logprobs", rows=16, vocab=131071, dtype="f32", scale=1.25, top=20, pad=0, banned=0.1),
        # the backward pass of the loss of a step's tokens
        dict(name="logprobs_grad_step", op="logprobs_grad", rows=8192, vocab=32000, dtype="bf16", scale=1.0, pad=100, entropy=False),
        # a byte-level vocabulary, many tokens, odd rows, with a bonus on the entropy
        dict(name="logprobs_grad_bytes", op="logprobs_grad", rows=65521, vocab=257, dtype="bf16", scale=0.8, pad=1000, entropy=True),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm; half of them multiples of 8 where that is in the range."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if v >= 16 and rng.random() < 0.5:
        v -= v % 8
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["dropout", "norm_block", "norm_block", "norm_grad", "norm_grad", "logprobs", "logprobs", "logprobs_grad"])
    kind = rng.choice(["bf16", "bf16", "f32"])
    if op == "dropout":
        return dict(op=op, rows=_log(rng, 1, 8192), cols=_log(rng, 8, 8192), dtype=kind, p=rng.choice([0.1, 0.2, 0.5, round(rng.uniform(0.01, 0.9), 3)]),
                    residual=rng.random() < 0.5)
    if op in ("norm_block", "norm_grad"):
        join = rng.random() < 0.75
        return dict(op=op, rows=_log(rng, 1, 8192), d=_log(rng, 16, 8192), kind=rng.choice(["layer", "rms"]), stream=kind,
                    block=rng.choice(["bf16", kind]), join=join, gate=rng.choice(["none", "vector", "matrix"]) if join else "none")
    vocab = _log(rng, 32, 131072)
    case = dict(op=op, rows=_log(rng, 1, min(65536, 8192 * 32000 // vocab // SIZE[kind] * 2)), vocab=vocab, dtype=kind, scale=rng.choice([1.0, 1.0, 0.8, 1.25]), pad=0)
    if op == "logprobs":
        return dict(case, top=rng.choice([0, 1, 5, 8, 20]), banned=rng.choice([0.0, 0.0, 0.1]))
    return dict(case, entropy=rng.random() < 0.4)


def work(case):
    op = case["op"]
    if op == "dropout":
        n, s = case["rows"] * case["cols"], SIZE[case["dtype"]]
        return {"bytes": n * s * (3 if case["residual"] else 2), "flops": 2 * n}
    if op in ("norm_block", "norm_grad"):
        n, x, f = case["rows"] * case["d"], SIZE[case["stream"]], SIZE[case["block"]]
        gates = 4 * case["d"] if case["gate"] == "vector" else n * f if case["gate"] == "matrix" else 0
        if op == "norm_block":  # the norm's parameters and the kept numbers too
            b = n * (2 * x + 2 * f) + gates + 16 * case["d"] if case["join"] else n * (x + f) + 8 * case["d"]
            return {"bytes": b + 16 * case["rows"], "flops": (18 if case["join"] else 8) * n}
        b = n * (3 * x + 3 * f) + 2 * gates + 32 * case["d"] if case["join"] else n * (3 * x + f) + 16 * case["d"]
        return {"bytes": b + 16 * case["rows"], "flops": (34 if case["join"] else 14) * n}
    n, s = case["rows"] * case["vocab"], SIZE[case["dtype"]]
    if op == "logprobs":
        return {"bytes": n * s + case["rows"] * (8 + 12 + 12 * case["top"]), "flops": 6 * n}
    return {"bytes": 2 * n * s + case["rows"] * 24, "flops": 6 * n}


# ---------------------------------------------------------------------------
# inputs


def _normal(g, *shape, s=1.0, m=0.0, dtype=F32):
    return (torch.randn(*shape, generator=g, device="cuda") * s + m).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op = case["op"]
    s = dict(case=case)
    if op == "dropout":
        s["x"] = _normal(g, case["rows"], case["cols"], dtype=TYPES[case["dtype"]])
        s["residual"] = _normal(g, case["rows"], case["cols"], dtype=TYPES[case["dtype"]]) if case["residual"] else None
        s["seed"] = (seed * 0x9E3779B97F4A7C15 + 12345) % 2 ** 64  # the run's seed; the call's site and its batch's first row beside it
        s["site"], s["first_row"] = 5, 3 * case["rows"]
    elif op in ("norm_block", "norm_grad"):
        rows, d, stream, block = case["rows"], case["d"], TYPES[case["stream"]], TYPES[case["block"]]
        s["x"] = _normal(g, rows, d, s=1.5, dtype=stream)
        s["alpha"], s["beta"] = (1.0, 1.0) if case["kind"] == "layer" else (0.875, 0.5)
        s["pre"] = (_normal(g, d, s=0.1, m=1.0), _normal(g, d, s=0.1) if case["kind"] == "layer" else None)
        s["f"] = s["post"] = s["gate"] = None
        if case["join"]:
            s["f"] = _normal(g, rows, d, s=0.5, m=0.1, dtype=block)
            s["post"] = (_normal(g, d, s=0.1, m=1.0), _normal(g, d, s=0.1) if case["kind"] == "layer" else None)
            if case["gate"] == "vector":
                s["gate"] = _normal(g, d, s=0.2, m=0.5)
            elif case["gate"] == "matrix":
                s["gate"] = torch.rand(rows, d, generator=g, device="cuda").to(block)
        if op == "norm_grad":  # x is the joined stream here, and its norm's input
            s["dh"] = _normal(g, rows, d, s=1e-2, dtype=block)
            s["dx"] = _normal(g, rows, d, s=1e-2, dtype=stream)
            s["kept"] = torch.zeros(rows, 4, device="cuda")
            if case["join"]:
                s["kept"][:, :2] = torch.cat(_moments(s["f"].float(), case["kind"]), 1)
            s["kept"][:, 2:] = torch.cat(_moments(s["x"].float(), case["kind"]), 1)
    else:
        rows, vocab = case["rows"], case["vocab"]
        z = _normal(g, rows, vocab, s=2.5)
        s["ids"] = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
        sure = torch.rand(rows, generator=g, device="cuda") * 12  # a model that has learnt something
        z.scatter_add_(1, s["ids"].unsqueeze(1), sure.unsqueeze(1))
        if case.get("banned"):
            z[:, torch.rand(vocab, generator=g, device="cuda") < case["banned"]] = BANNED
        s["logits"] = z.to(TYPES[case["dtype"]])
        del z
        if case["pad"]:
            s["ids"][-case["pad"]:] = -1
        if op == "logprobs_grad":
            s["lse"], s["entropy"] = _distribution(s["logits"].float() * case["scale"])[:2]
            s["g"] = _normal(g, rows, s=1.0 / rows, m=-1.0 / rows)
            s["gh"] = _normal(g, rows, s=0.01 / rows) if case["entropy"] else None
    return s


# ---------------------------------------------------------------------------
# the plain forms


def _mul32(a, b):
    """The high and the low word of the product of 32-bit numbers held in 64 bits (b a constant)."""
    p = a * b  # wraps; the words of the unsigned product all the same
    return (p >> 32) & 0xFFFFFFFF, p & 0xFFFFFFFF


def _kept_mask(rows, cols, p, seed, site, first_row):
    """(where a value is kept, its scale)"""
    groups = -(-cols // 8)
    c0 = torch.arange(groups, device="cuda").expand(rows, groups)
    row = torch.arange(first_row, first_row + rows, device="cuda").unsqueeze(1).expand(rows, groups)
    c1, c2, c3 = torch.full_like(c0, site), row & 0xFFFFFFFF, row >> 32
    k0, k1 = seed & 0xFFFFFFFF, seed >> 32
    for _ in range(10):
        h0, l0 = _mul32(c0, 0xD2511F53)
        h1, l1 = _mul32(c2, 0xCD9E8D57)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    halves = [w for c in (c0, c1, c2, c3) for w in (c & 0xFFFF, c >> 16)]
    t = round(65536 * p)
    return (torch.stack(halves, 2) >= t).view(rows, groups * 8)[:, :cols], 65536 / (65536 - t) if t < 65536 else 0.0


def _moments(v, kind):
    """m and rstd of each row, as columns"""
    m = v.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(v[:, :1])
    return m, ((v - m).square().mean(1, keepdim=True) + EPS).rsqrt()


def _normed(v, m, rstd, norm):
    y = (v - m) * rstd * norm[0]
    return y if norm[1] is None else y + norm[1]


def _distribution(z):
    """(lse, entropy, log probabilities) of each row"""
    top = z.amax(1, keepdim=True)
    logp = z - top
    logp = logp - torch.exp(logp).sum(1, keepdim=True).log()
    p = torch.exp(logp)
    h = -torch.where(p > 0, p * logp, 0.0).sum(1)
    first = logp.argmax(1, keepdim=True)
    return (top - logp.gather(1, first)).squeeze(1), h, logp


def _alternatives(logits, logp, count):
    """The most likely tokens and their log probabilities, the lowest index first among equals; -1 where no possible token is left."""
    left, ids, values = logits.clone(), [], []
    for _ in range(count):
        top, at = left.max(1, keepdim=True)
        none = top == BANNED
        ids.append(torch.where(none, -1, at))
        values.append(torch.where(none, BANNED, logp.gather(1, at)))
        left.scatter_(1, at, BANNED)
    return torch.cat(ids, 1), torch.cat(values, 1)


def _plain(s):
    c, op = s["case"], s["case"]["op"]
    if op == "dropout":
        keep, scale = _kept_mask(c["rows"], c["cols"], c["p"], s["seed"], s["site"], s["first_row"])
        y = torch.where(keep, s["x"].float() * scale, 0.0)
        return (y if s["residual"] is None else y + s["residual"].float()).to(s["x"].dtype)
    if op == "norm_block":
        x = s["x"]
        kept = torch.zeros(c["rows"], 4, device="cuda")
        if c["join"]:
            f = s["f"].float()
            m, rstd = _moments(f, c["kind"])
            kept[:, 0:1], kept[:, 1:2] = m, rstd
            y = _normed(f, m, rstd, s["post"])
            if s["gate"] is not None:
                y = y * s["gate"].float()
            x = (s["alpha"] * x.float() + s["beta"] * y).to(x.dtype)
        v = x.float()
        m, rstd = _moments(v, c["kind"])
        kept[:, 2:3], kept[:, 3:4] = m, rstd
        out = {"h": _normed(v, m, rstd, s["pre"]).to(TYPES[c["block"]]), "kept": kept}
        return dict(out, x=x) if c["join"] else out
    if op == "norm_grad":
        layer = c["kind"] == "layer"
        kept = s["kept"]
        dh, xh = s["dh"].float(), (s["x"].float() - kept[:, 2:3]) * kept[:, 3:4]
        v = dh * s["pre"][0]
        inner = v - xh * (v * xh).mean(1, keepdim=True)
        if layer:
            inner = inner - v.mean(1, keepdim=True)
        full = s["dx"].float() + kept[:, 3:4] * inner
        out = {"pre_gain": (dh * xh).sum(0)}
        if layer:
            out["pre_bias"] = dh.sum(0)
        if not c["join"]:
            return dict(out, dx=full.to(s["x"].dtype))
        out["dx"] = (s["alpha"] * full).to(s["x"].dtype)
        full = s["beta"] * full
        fh = (s["f"].float() - kept[:, 0:1]) * kept[:, 1:2]
        if s["gate"] is not None:
            n = fh * s["post"][0]
            n = full * (n if s["post"][1] is None else n + s["post"][1])
            out["gate"] = n.sum(0) if c["gate"] == "vector" else n.to(s["gate"].dtype)
            full = full * s["gate"].float()
        out["post_gain"] = (full * fh).sum(0)
        if layer:
            out["post_bias"] = full.sum(0)
        w = full * s["post"][0]
        inner = w - fh * (w * fh).mean(1, keepdim=True)
        if layer:
            inner = inner - w.mean(1, keepdim=True)
        out["df"] = (kept[:, 1:2] * inner).to(TYPES[c["block"]])
        return out
    z = s["logits"].float() * c["scale"]
    ids = s["ids"]
    given = (ids >= 0).unsqueeze(1)
    if op == "logprobs":
        lse, h, logp = _distribution(z)
        picked = logp.gather(1, ids.clamp(min=0).unsqueeze(1))
        out = {"logp": torch.where(given, picked, 0.0).squeeze(1), "lse": lse, "entropy": h}
        if c["top"]:
            out["top_ids"], out["top_logp"] = _alternatives(s["logits"], logp, c["top"])
        return out
    logp = z - s["lse"].unsqueeze(1)
    p = torch.exp(logp)
    g = torch.where(given.squeeze(1), s["g"], 0.0).unsqueeze(1)
    d = -g * p
    d.scatter_add_(1, ids.clamp(min=0).unsqueeze(1), g)
    if s["gh"] is not None:
        d = d - s["gh"].unsqueeze(1) * torch.where(p > 0, p * (logp + s["entropy"].unsqueeze(1)), 0.0)
    return (d * c["scale"]).to(s["logits"].dtype)


def _own(s):
    import gradient_ring_all_gb300 as ra
    c, op = s["case"], s["case"]["op"]
    if op == "dropout":
        return ra.ra_dropout(s["x"], c["p"], s["seed"], site=s["site"], first_row=s["first_row"], residual=s["residual"])
    if op in ("norm_block", "norm_grad"):
        pre = ra.Norm(*s["pre"], kind=c["kind"], eps=EPS)
        post = ra.Norm(*s["post"], kind=c["kind"], eps=EPS) if c["join"] else None
        if op == "norm_block":
            x, h, kept = ra.ra_norm_block(s["x"], s["f"], post=post, gate=s["gate"], alpha=s["alpha"], beta=s["beta"], pre=pre, dtype=TYPES[c["block"]])
            return {"x": x, "h": h, "kept": kept} if c["join"] else {"h": h, "kept": kept}
        alpha, beta = (s["alpha"], s["beta"]) if c["join"] else (1.0, 1.0)
        d = ra.ra_norm_block_grad(s["dh"], s["x"], s["kept"], f=s["f"], post=post, gate=s["gate"], alpha=alpha, beta=beta, pre=pre, dx=s["dx"])
        out = {"dx": d.dx, "df": d.df, "gate": d.gate, "post_gain": d.post_gain, "post_bias": d.post_bias, "pre_gain": d.pre_gain, "pre_bias": d.pre_bias}
        return {k: t for k, t in out.items() if t is not None}
    if op == "logprobs":
        r = ra.ra_logprobs(s["logits"], s["ids"], scale=c["scale"], entropy=True, top=c["top"])
        out = {"logp": r.logp, "lse": r.lse, "entropy": r.entropy}
        return dict(out, top_ids=r.top_ids, top_logp=r.top_logp) if c["top"] else out
    entropy = dict(entropy=s["entropy"], grad_entropy=s["gh"]) if c["entropy"] else {}
    return ra.ra_logprobs_grad(s["logits"], s["ids"], s["lse"], s["g"], scale=c["scale"], **entropy)


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# the definitions, in 64 bits


def _philox_halves(rows, groups, seed, site, first_row):
    """The 16-bit numbers of each row's groups, on the host."""
    low, half = np.uint64(0xFFFFFFFF), np.uint64(32)
    row = (np.arange(rows, dtype=np.uint64) + np.uint64(first_row))[:, None]
    ctr = [np.arange(groups, dtype=np.uint64)[None, :] + 0 * row, np.uint64(site) + np.zeros((rows, groups), np.uint64), (row & low) + np.zeros((rows, groups), np.uint64),
           (row >> half) + np.zeros((rows, groups), np.uint64)]
    key = [seed % 2 ** 32, seed // 2 ** 32]
    for _ in range(10):
        a, b = ctr[0] * np.uint64(0xD2511F53), ctr[2] * np.uint64(0xCD9E8D57)
        ctr = [(b >> half) ^ ctr[1] ^ np.uint64(key[0]), b & low, (a >> half) ^ ctr[3] ^ np.uint64(key[1]), a & low]
        key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
    words = np.stack(ctr, 2).astype("<u4")
    return words.view("<u2").reshape(rows, groups * 8)


def _norm64(v, kind, norm):
    centre = v.mean(1, keepdim=True) if kind == "layer" else 0.0
    size = torch.sqrt(torch.sum((v - centre) ** 2, 1, keepdim=True) / v.shape[1] + EPS)
    unit = (v - centre) / size
    y = unit * norm[0].double()
    if norm[1] is not None:
        y = y + norm[1].double()
    stats = torch.cat([torch.zeros_like(size) + centre, 1 / size], 1)
    return y, unit, size, stats


def _norm_back64(v, unit, size, kind):
    """The gradient through (v - m) / size, `v` that of the unit row."""
    out = v - unit * torch.sum(v * unit, 1, keepdim=True) / v.shape[1]
    if kind == "layer":
        out = out - torch.sum(v, 1, keepdim=True) / v.shape[1]
    return out / size


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "dropout":
        rows, cols = case["rows"], case["cols"]
        t = round(65536 * case["p"])
        u = _philox_halves(rows, -(-cols // 8), s["seed"], s["site"], s["first_row"])[:, :cols]
        keep = torch.from_numpy(u >= t).cuda()
        y = s["x"].double() * keep * (65536 / (65536 - t))
        return y if s["residual"] is None else y + s["residual"].double()
    if op == "norm_block":
        x, stats = s["x"].double(), torch.zeros(case["rows"], 2, dtype=torch.float64, device="cuda")
        out = {}
        if case["join"]:
            y, _, _, stats = _norm64(s["f"].double(), case["kind"], s["post"])
            x = s["alpha"] * x + s["beta"] * (y if s["gate"] is None else s["gate"].double() * y)
            out["x"] = x
            x = x.to(s["x"].dtype).double()  # the norm is that of the stream as it is stored
        h, _, _, more = _norm64(x, case["kind"], s["pre"])
        return dict(out, h=h, kept=torch.cat([stats, more], 1))
    if op == "norm_grad":
        layer = case["kind"] == "layer"
        dh = s["dh"].double()
        _, unit, size, _ = _norm64(s["x"].double(), case["kind"], s["pre"])
        full = s["dx"].double() + _norm_back64(dh * s["pre"][0].double(), unit, size, case["kind"])
        out = {"pre_gain": torch.sum(dh * unit, 0)}
        if layer:
            out["pre_bias"] = torch.sum(dh, 0)
        if not case["join"]:
            return dict(out, dx=full)
        out["dx"] = s["alpha"] * full
        y, unit, size, _ = _norm64(s["f"].double(), case["kind"], s["post"])
        u = s["beta"] * full
        if s["gate"] is not None:
            out["gate"] = torch.sum(u * y, 0) if case["gate"] == "vector" else u * y
            u = u * s["gate"].double()
        out["post_gain"] = torch.sum(u * unit, 0)
        if layer:
            out["post_bias"] = torch.sum(u, 0)
        out["df"] = _norm_back64(u * s["post"][0].double(), unit, size, case["kind"])
        return out
    z = s["logits"].double() * case["scale"]
    rows = torch.arange(case["rows"], device="cuda")
    given = s["ids"] >= 0
    lse = torch.logsumexp(z, 1)
    if op == "logprobs":
        picked = torch.where(given, z[rows, s["ids"].clamp(min=0)] - lse, 0.0)
        p = torch.exp(z - lse.unsqueeze(1))
        out = {"logp": picked, "lse": lse, "entropy": lse - torch.sum(torch.where(p > 0, p * z, 0.0), 1)}
        if case["top"]:
            del p
            order = torch.sort(s["logits"], dim=1, descending=True, stable=True)
            ids, top = order.indices[:, :case["top"]], order.values[:, :case["top"]]
            out["top_ids"] = torch.where(top == BANNED, -1, ids)
            out["top_logp"] = top.double() * case["scale"] - lse.unsqueeze(1)
        return out
    p = torch.exp(z - lse.unsqueeze(1))
    g = torch.where(given, s["g"].double(), 0.0)
    d = p * -g.unsqueeze(1)
    d[rows, s["ids"].clamp(min=0)] += g
    if s["gh"] is not None:
        t = torch.where(p > 0, p * z, 0.0)
        d -= s["gh"].double().unsqueeze(1) * (t - p * torch.sum(t, 1, keepdim=True))
    return d * case["scale"]
