"""Plain references in 64 bits of the operators between a step's products, and
the error bounds their tests hold the kernels to.

u = 2^-24 is binary32's unit roundoff.  Sums are trees: a value of a row passes
through fewer than 64 additions (16 in a thread, 5 of a warp's shuffles, 16
warps, 8 blocks), so a row's sum is off by at most 64 u times the sum of the
magnitudes.  A value of a column passes through at most 128 in the tests' sizes
(rows / 152 in a block, at most 8 groups, 304 / 8 + 8 parts).

The norms' results are compared with MAGNITUDE * 512 u, where MAGNITUDE is the
result's own formula with every term replaced by its magnitude and every sum by
the sum of magnitudes, and where a normed value (v - m) * rstd counts as
rstd * (|v| + mean |v|), which bounds it and its rounding's source.  Each
elementary operation adds at most u of its magnitude, a row's sum 64 u, a
column's 128 u, rsqrt 4 u; the longest chain (a column's sum of a product that
holds two rows' sums and the moments of two norms, each of which is a sum and an
rstd) adds up to 4 * 64 + 128 + 2 * 40 + 20 < 512."""
from __future__ import annotations

import numpy as np
import torch

U = 2.0 ** -24
CHAIN = 512 * U


def half_step(dtype) -> float:
    """The most a rounding to the type is off by, relative to the value."""
    return torch.finfo(dtype).eps / 2


# ---------------------------------------------------------------------------
# dropout

M0, M1, W0, W1 = 0xD2511F53, 0xCD9E8D57, 0x9E3779B9, 0xBB67AE85


def philox(counter, key):
    """Philox4x32-10 in Python's whole numbers: four words of a counter of four and a key of two."""
    c, k = list(counter), list(key)
    for _ in range(10):
        a, b = M0 * c[0], M1 * c[2]
        c = [(b >> 32) ^ c[1] ^ k[0], b % 2 ** 32, (a >> 32) ^ c[3] ^ k[1], a % 2 ** 32]
        k = [(k[0] + W0) % 2 ** 32, (k[1] + W1) % 2 ** 32]
    return c


def keep_mask(rows, cols, p, seed, site=0, first_row=0):
    """Where a value is kept, on the host: the same by 64-bit arrays."""
    groups = -(-cols // 8)
    full = lambda v: np.broadcast_to(np.asarray(v, dtype=np.uint64), (rows, groups))  # noqa: E731
    low, h = np.uint64(0xFFFFFFFF), np.uint64(32)
    row = (np.arange(rows, dtype=np.uint64) + np.uint64(first_row))[:, None]
    c = [full(np.arange(groups, dtype=np.uint64)[None, :]), full(np.uint64(site)), full(row & low), full(row >> h)]
    k0, k1 = seed % 2 ** 32, seed >> 32
    for _ in range(10):
        a, b = c[0] * np.uint64(M0), c[2] * np.uint64(M1)
        c = [(b >> h) ^ c[1] ^ np.uint64(k0), b & low, (a >> h) ^ c[3] ^ np.uint64(k1), a & low]
        k0, k1 = (k0 + W0) % 2 ** 32, (k1 + W1) % 2 ** 32
    halves = np.stack([w >> np.uint64(16 * i) & np.uint64(0xFFFF) for w in c for i in (0, 1)], 2).reshape(rows, groups * 8)
    return torch.from_numpy(halves[:, :cols] >= round(65536 * p))


# ---------------------------------------------------------------------------
# norms


def _moments(v, kind, eps):
    m = v.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(v[:, :1])
    return m, ((v - m).square().mean(1, keepdim=True) + eps).rsqrt()


def _params(n):
    return (1.0 if n.gain is None else n.gain.double()), (0.0 if n.bias is None else n.bias.double())


def _abs(v):
    return v.abs() if torch.is_tensor(v) else abs(v)


def _norm64(v, n):
    """(result, its magnitude, unit row, the unit row's magnitude, m, rstd)"""
    m, rstd = _moments(v, n.kind, n.eps)
    g, b = _params(n)
    unit = (v - m) * rstd
    size = rstd * (v.abs() + v.abs().mean(1, keepdim=True))
    return unit * g + b, size * _abs(g) + _abs(b), unit, size, m, rstd


def join64(x, f, post, gate, alpha, beta):
    """(x', its magnitude) before its rounding"""
    y, size = (f.double(), f.double().abs()) if post is None else _norm64(f.double(), post)[:2]
    if gate is not None:
        y, size = y * gate.double(), size * gate.double().abs()
    return alpha * x.double() + beta * y, abs(alpha) * x.double().abs() + abs(beta) * size


def grads64(dh, x, f, post, gate, alpha, beta, pre, dx):
    """{name: (gradient, its magnitude)}"""
    out = {}
    full = torch.zeros_like(x, dtype=torch.float64) if dx is None else dx.double()
    big = full.abs()
    if pre is not None:
        _, _, unit, size, _, rstd = _norm64(x.double(), pre)
        g, _ = _params(pre)
        d = dh.double()
        out["pre_gain"] = (d * unit).sum(0), (d.abs() * size).sum(0)
        out["pre_bias"] = d.sum(0), d.abs().sum(0)
        v = d * g
        t = v - unit * (v * unit).mean(1, keepdim=True)
        s = v.abs() + size * (v.abs() * size).mean(1, keepdim=True)
        if pre.kind == "layer":
            t, s = t - v.mean(1, keepdim=True), s + v.abs().mean(1, keepdim=True)
        full, big = full + rstd * t, big + rstd * s
    if f is None:
        out["dx"] = full, big
        return out
    out["dx"] = alpha * full, abs(alpha) * big
    u, big = beta * full, abs(beta) * big
    if post is None:
        n = unit = f.double()
        n_size = size = unit.abs()
    else:
        n, n_size, unit, size, _, rstd = _norm64(f.double(), post)
    if gate is not None:
        t, s = u * n, big * n_size
        out["gate"] = (t.sum(0), s.sum(0)) if gate.dim() == 1 else (t, s)
        u, big = u * gate.double(), big * gate.double().abs()
    if post is None:
        out["df"] = u, big
        return out
    out["post_gain"] = (u * unit).sum(0), (big * size).sum(0)
    out["post_bias"] = u.sum(0), big.sum(0)
    g, _ = _params(post)
    w, big = u * g, big * _abs(g)
    t = w - unit * (w * unit).mean(1, keepdim=True)
    s = big + size * (big * size).mean(1, keepdim=True)
    if post.kind == "layer":
        t, s = t - w.mean(1, keepdim=True), s + big.mean(1, keepdim=True)
    out["df"] = rstd * t, rstd * s
    return out


# ---------------------------------------------------------------------------
# log probabilities


def distribution64(logits, scale):
    """(z, m, log s, entropy, p) of softmax(scale * logits): m a row's largest z and s the sum of exp(z - m), so that values far
    from zero lose nothing.  A row in which no token can be has m 0, log s minus infinity, entropy and p 0."""
    z = logits.double() * scale
    m = z.amax(1) if z.shape[1] else torch.full(z.shape[:1], -float("inf"), dtype=torch.float64, device=z.device)
    m = torch.where(m == -float("inf"), 0.0, m)
    y = z - m.unsqueeze(1)
    log_s = torch.exp(y).sum(1).log()
    lp = y - log_s.unsqueeze(1)
    p = torch.where((log_s == -float("inf")).unsqueeze(1), 0.0, torch.exp(lp))
    t = torch.where(z == -float("inf"), 0.0, p * lp)
    return z, m, log_s, -t.sum(1), p


def alternatives64(logits, count):
    """The `count` likeliest tokens of each row by value and index, on the host: -1 where none is left, and throughout a row with
    a NaN or plus infinity."""
    rows, vocab = logits.shape
    z = logits.float().cpu().numpy()
    out = np.full((rows, count), -1, dtype=np.int64)
    for r in range(rows):
        row = z[r] + np.float32(0)
        if np.isnan(row).any() or (row == np.inf).any():
            continue
        order = np.lexsort((np.arange(vocab), -row.astype(np.float64)))
        order = order[~(row[order] == -np.inf)][:count]
        out[r, :len(order)] = order
    return torch.from_numpy(out)
