"""The operators of a data-parallel training step around the gradient ring:
what they compute, and the cases they are measured on.

Five operators produce the gradients that the ring averages:

- ``lookup``     rows of an embedding table, scaled
- ``table_grad`` the table's gradient, summed over the tokens of each id
- ``linear``     act(x @ w + bias) + residual, with the pre-activation kept in 8 bits if asked
- ``backward``   that layer's gradients from the 8-bit checkpoint of its input:
                 dz = (dy @ w^T) * act'(z), dw = act(z)^T @ dy, db = the column sums of dy
- ``checkpoint`` an activation kept in 8 bits and restored

``run`` computes each in elementary torch operations in 32 bits, or, with
``own`` true, through the package's calls on the same inputs.  ``exact`` is the
definition in 64 bits.

An activation in 8 bits: groups of 32 neighbours of a row share one power of
two.  With E the exponent of the group's largest magnitude (one more if that
magnitude is so near the next power that it would round to 128 steps), the
step is 2^(E-6) and every value is the nearest whole number of steps, -127 to
127.  The step is held as the byte E - 6 + 127, at least 1.

Sizes: the Transformer of the package's workloads (d 2048, ffn 8192, vocabulary
32000, 8192 tokens a step), ResNet-18's 512-wide head, and odd ones.
"""
from __future__ import annotations

import math

import torch

own = False

GROUP = 32
BF16, F32 = torch.bfloat16, torch.float32
TYPES = {"bf16": BF16, "f32": F32}
SIZE = {"bf16": 2, "f32": 4}


def listed():
    return [
        # the step's token ids through the input embedding, scaled by sqrt(d)
        dict(name="lookup_step", op="lookup", tokens=16384, vocab=32000, d=2048, dtype="bf16", pad=0),
        # a handful of tokens of a small binary32 table, odd width: latency
        dict(name="lookup_few", op="lookup", tokens=37, vocab=1000, d=509, dtype="f32", pad=3),
        # the input embedding's gradient into a binary32 gradient row; word frequencies fall as 1/rank
        dict(name="table_grad_step", op="table_grad", tokens=8192, vocab=32000, d=2048, dtype="bf16", out="f32", pad=100),
        # a byte-level table: few ids, each thousands of times; odd width
        dict(name="table_grad_bytes", op="table_grad", tokens=65521, vocab=257, d=1022, dtype="bf16", out="bf16", pad=0),
        # the ffn's first product with its activation, the pre-activation kept in 8 bits for the backward pass
        dict(name="linear_ffn_up", op="linear", m=8192, k=2048, n=8192, act="gelu", residual=False, save=True, out="bf16"),
        # the ffn's second product, added to the residual stream
        dict(name="linear_ffn_down", op="linear", m=8192, k=8192, n=2048, act="none", residual=True, save=False, out="bf16"),
        # one token through the ffn's first product
        dict(name="linear_token", op="linear", m=1, k=2048, n=8192, act="gelu", residual=False, save=False, out="bf16"),
        # a ragged batch through a layer whose rows share no 16-byte boundary, binary32 result
        dict(name="linear_ragged", op="linear", m=1111, k=1999, n=1001, act="silu", residual=True, save=False, out="f32"),
        # the backward pass of the ffn's second product from the 8-bit pre-activation
        dict(name="backward_ffn", op="backward", m=8192, k=8192, n=2048, act="gelu", dtype="bf16"),
        # a ragged micro-batch of a 512-wide layer, binary32 weight gradient
        dict(name="backward_ragged", op="backward", m=777, k=1003, n=512, act="none", dtype="f32"),
        # the ffn's hidden activation, kept and restored
        dict(name="checkpoint_ffn", op="checkpoint", m=8192, k=8192, dtype="bf16"),
        # a small odd one in binary32: the last group of each row is cut short
        dict(name="checkpoint_odd", op="checkpoint", m=333, k=1001, dtype="f32"),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm; half of them multiples of 8 where that is in the range."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if v >= 16 and rng.random() < 0.5:
        v -= v % 8
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["lookup", "table_grad", "linear", "linear", "backward", "backward", "checkpoint"])
    if op == "lookup":
        return dict(op=op, tokens=_log(rng, 1, 16384), vocab=_log(rng, 200, 32000), d=_log(rng, 64, 2048), dtype=rng.choice(["bf16", "f32"]), pad=0)
    if op == "table_grad":
        return dict(op=op, tokens=_log(rng, 1, 32768), vocab=_log(rng, 200, 32000), d=_log(rng, 64, 2048), dtype=rng.choice(["bf16", "f32"]),
                    out=rng.choice(["bf16", "f32"]), pad=0)
    if op == "linear":
        return dict(op=op, m=_log(rng, 1, 8192), k=_log(rng, 64, 4096), n=_log(rng, 64, 8192), act=rng.choice(["none", "relu", "gelu", "silu"]),
                    residual=rng.random() < 0.5, save=rng.random() < 0.3, out=rng.choice(["bf16", "bf16", "f32"]))
    if op == "backward":
        act = rng.choice(["none", "none", "relu", "gelu", "silu"])
        return dict(op=op, m=_log(rng, 1, 8192), k=_log(rng, 64, 4096), n=_log(rng, 64, 4096), act=act, dtype="bf16" if act != "none" else rng.choice(["bf16", "f32"]))
    return dict(op=op, m=_log(rng, 1, 8192), k=_log(rng, 64, 8192), dtype=rng.choice(["bf16", "f32"]))


def work(case):
    op = case["op"]
    if op == "lookup":
        t, d, s = case["tokens"], case["d"], SIZE[case["dtype"]]
        return {"bytes": (min(t, case["vocab"]) + t) * d * s + 8 * t, "flops": t * d}
    if op == "table_grad":
        t, d = case["tokens"], case["d"]
        return {"bytes": t * d * SIZE[case["dtype"]] + case["vocab"] * d * SIZE[case["out"]] + 8 * t, "flops": t * d}
    m, k = case["m"], case["k"]
    kept = m * (k + -(-k // GROUP))  # k values and their groups' bytes
    if op == "checkpoint":
        return {"bytes": 2 * m * k * SIZE[case["dtype"]] + 2 * kept, "flops": 3 * m * k}
    n = case["n"]
    if op == "linear":
        b = 2 * (m * k + k * n) + 4 * n + m * n * SIZE[case["out"]]
        b += 2 * m * n if case["residual"] else 0
        b += m * (n + -(-n // GROUP)) if case["save"] else 0
        return {"bytes": b, "flops": 2 * m * k * n}
    return {"bytes": 2 * m * n + 2 * k * n + kept + 2 * m * k + k * n * SIZE[case["dtype"]] + 4 * n, "flops": 4 * m * k * n}


def _ids(g, count, vocab, pad):
    """Token ids whose frequency falls as 1/rank; the last `pad` are -1 (padding)."""
    w = 1.0 / torch.arange(1, vocab + 1, device="cuda", dtype=torch.float64)
    edges = torch.cumsum(w, 0) / w.sum()
    ids = torch.searchsorted(edges, torch.rand(count, generator=g, device="cuda", dtype=torch.float64)).clamp_(max=vocab - 1)
    if pad:
        ids[-pad:] = -1
    return ids


def _normal(g, *shape, s=1.0, dtype=BF16):
    return (torch.randn(*shape, generator=g, device="cuda") * s).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op = case["op"]
    s = dict(case=case)
    if op == "lookup":
        s["table"] = _normal(g, case["vocab"], case["d"], s=0.02, dtype=TYPES[case["dtype"]])
        s["ids"] = _ids(g, case["tokens"], case["vocab"], case["pad"])
    elif op == "table_grad":
        s["grad"] = _normal(g, case["tokens"], case["d"], s=1e-2, dtype=TYPES[case["dtype"]])
        s["ids"] = _ids(g, case["tokens"], case["vocab"], case["pad"])
    elif op == "checkpoint":
        s["x"] = _normal(g, case["m"], case["k"], dtype=TYPES[case["dtype"]])
    elif op == "linear":
        m, k, n = case["m"], case["k"], case["n"]
        s["x"] = _normal(g, m, k)
        s["w"] = _normal(g, k, n, s=k ** -0.5)
        s["bias"] = _normal(g, n, s=0.1, dtype=F32)
        s["residual"] = _normal(g, m, n) if case["residual"] else None
    else:
        m, k, n = case["m"], case["k"], case["n"]
        s["dy"] = _normal(g, m, n, s=1e-2)
        s["w"] = _normal(g, k, n, s=k ** -0.5)
        s["q"], s["e"] = _pack(_normal(g, m, k))
    return s


# ---------------------------------------------------------------------------
# the plain forms


def _pack(x):
    """The 8-bit form of a matrix: q int8 [rows, columns rounded up to groups], e uint8 [rows, groups]."""
    rows, cols = x.shape
    x = torch.nn.functional.pad(x.float(), (0, -cols % GROUP)).view(rows, -1, GROUP)
    top = x.abs().amax(2, keepdim=True)
    e = (((top.view(torch.int32) + 0x10000) >> 23) - 6).clamp(min=1)
    q = torch.round(x * ((254 - e) << 23).view(F32))
    return q.to(torch.int8).view(rows, -1), e.to(torch.uint8).view(rows, -1)


def _values(q, e, cols):
    """What the 8-bit form stands for, in binary32."""
    rows = q.shape[0]
    step = (e.to(torch.int32) << 23).view(F32)
    return (q.float().view(rows, -1, GROUP) * step.unsqueeze(2)).view(rows, -1)[:, :cols]


def _act(z, act):
    if act == "relu":
        return torch.clamp(z, min=0)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * 2 ** -0.5))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * 2 ** -0.5)) + z * torch.exp(-0.5 * z * z) * (2 * math.pi) ** -0.5
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    return torch.ones_like(z)


def _plain(s):
    c, op = s["case"], s["case"]["op"]
    if op == "lookup":
        ids = s["ids"]
        rows = s["table"].float()[ids.clamp(min=0)] * c["d"] ** 0.5
        return torch.where((ids >= 0).unsqueeze(1), rows, 0.0).to(s["table"].dtype)
    if op == "table_grad":
        ids = s["ids"]
        keep = (ids >= 0).unsqueeze(1)
        out = torch.zeros(c["vocab"], c["d"], device="cuda")
        out.index_add_(0, ids.clamp(min=0), torch.where(keep, s["grad"].float(), 0.0))
        return (out * c["d"] ** 0.5).to(TYPES[c["out"]])
    if op == "checkpoint":
        return _values(*_pack(s["x"]), c["k"]).to(s["x"].dtype)
    if op == "linear":
        z = s["x"].float() @ s["w"].float() + s["bias"]
        y = _act(z, c["act"])
        if s["residual"] is not None:
            y = y + s["residual"].float()
        y = y.to(TYPES[c["out"]])
        return {"y": y, "kept": _values(*_pack(z), c["n"]).to(BF16)} if c["save"] else {"y": y}
    z = _values(s["q"], s["e"], c["k"])
    dy = s["dy"].float()
    dz = (dy @ s["w"].float().t()) * _slope(z, c["act"])
    return {"dz": dz.to(BF16), "dw": (_act(z, c["act"]).t() @ dy).to(TYPES[c["dtype"]]), "db": dy.sum(0)}


def _own(s):
    import gradient_ring_all_gb300 as ra
    c, op = s["case"], s["case"]["op"]
    if op == "lookup":
        return ra.ra_embedding_lookup(s["table"], s["ids"], scale=c["d"] ** 0.5)
    if op == "table_grad":
        return ra.ra_embedding_grad(s["grad"], s["ids"], c["vocab"], scale=c["d"] ** 0.5, dtype=TYPES[c["out"]])
    if op == "checkpoint":
        return ra.ra_checkpoint8_unpack(ra.ra_checkpoint8_pack(s["x"]), dtype=s["x"].dtype)
    if op == "linear":
        kept = ra.Checkpoint8(c["m"], c["n"]) if c["save"] else None
        y = ra.ra_linear(s["x"], s["w"], bias=s["bias"], act=c["act"], residual=s["residual"], save=kept, dtype=TYPES[c["out"]])
        return {"y": y, "kept": ra.ra_checkpoint8_unpack(kept)} if c["save"] else {"y": y}
    z = ra.Checkpoint8(c["m"], c["k"], q=s["q"], e=s["e"])
    dz = ra.ra_linear_dgrad(s["dy"], s["w"], saved=z, act=c["act"])
    dw, db = ra.ra_linear_wgrad(z, s["dy"], act=c["act"], dtype=TYPES[c["dtype"]], bias_grad=True)
    return {"dz": dz, "dw": dw, "db": db}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# the definitions, in 64 bits


def _steps64(x):
    """Each value's step of the 8-bit form, in 64 bits."""
    rows, cols = x.shape
    top = torch.nn.functional.pad(x.abs(), (0, -cols % GROUP)).view(rows, -1, GROUP).amax(2)
    half, power = torch.frexp(top)  # top = half * 2^power, half in [0.5, 1)
    power = power.double() - 1 + (2 * half >= 255 / 128).double()
    step = torch.exp2(torch.where(top > 0, (power - 6).clamp(min=-126), -126.0))
    return step.repeat_interleave(GROUP, 1)[:, :cols]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "lookup":
        ids = s["ids"]
        out = math.sqrt(case["d"]) * s["table"].double().index_select(0, ids.clamp(min=0))
        out[ids < 0] = 0
        return out
    if op == "table_grad":
        ids = s["ids"]
        keep = ids >= 0
        out = torch.zeros(case["vocab"], case["d"], dtype=torch.float64, device="cuda")
        return out.index_add_(0, ids[keep], s["grad"].double()[keep]) * math.sqrt(case["d"])
    if op == "checkpoint":
        x = s["x"].double()
        step = _steps64(x)
        return torch.round(x / step) * step
    if op == "linear":
        z = s["x"].double() @ s["w"].double() + s["bias"].double()
        y = z
        if case["act"] == "relu":
            y = torch.where(z > 0, z, 0.0)
        elif case["act"] == "gelu":
            y = z * (0.5 * torch.special.erfc(-z / math.sqrt(2)))
        elif case["act"] == "silu":
            y = z * torch.sigmoid(z)
        if s["residual"] is not None:
            y = y + s["residual"].double()
        # the checkpoint is a rounding of z to 8 bits, as y's type is one to 16: both are given before that rounding
        return {"y": y, "kept": z} if case["save"] else {"y": y}
    k = case["k"]
    z = torch.ldexp(s["q"].double(), s["e"].double().repeat_interleave(GROUP, 1) - 127)[:, :k]
    a, slope = z, torch.ones_like(z)
    if case["act"] == "relu":
        slope = torch.heaviside(z, torch.zeros((), dtype=torch.float64, device="cuda"))
        a = z * slope
    elif case["act"] == "gelu":
        phi = 0.5 * torch.special.erfc(-z / math.sqrt(2))
        a, slope = z * phi, phi + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    elif case["act"] == "silu":
        p = torch.sigmoid(z)
        a, slope = z * p, p + z * p * (1 - p)
    dy = s["dy"].double()
    return {"dz": (dy @ s["w"].double().t()) * slope, "dw": a.t() @ dy, "db": dy.sum(0)}
