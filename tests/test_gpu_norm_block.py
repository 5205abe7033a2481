"""ra_norm_block and ra_norm_block_grad against plain forms in 64 bits
(block_reference.py derives the bounds)."""
from __future__ import annotations

import pytest
import torch

import gradient_ring_all_gb300 as ra
from block_reference import CHAIN, U, grads64, half_step, join64, _norm64
from operator_reference import Framed, check

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
TYPES = [(BF16, BF16), (F32, F32), (F32, BF16)]
SIZES = [(1, 1), (1, 8), (3, 31), (1, 2048), (130, 256), (41, 264), (65, 512), (9, 520), (300, 1024), (33, 1003), (17, 2047), (700, 2048), (12, 4096), (5, 4100),
         (6, 8192), (3, 8200), (2, 16384), (3, 20001), (2, 32768)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from gradient_ring_all_gb300 import build
    build.build()
    ra.load()


class _Case:
    """Inputs of one call, in frames."""

    def __init__(self, rows, d, stream, block, kind, gate, join=True, bias=True, lead=0, gap=0, param=F32, mean=0.3):
        g = torch.Generator(device="cuda").manual_seed(rows * 1000 + d)
        normal = lambda *s, m=0.0, k=1.0: torch.randn(*s, generator=g, device="cuda") * k + m  # noqa: E731
        frame = lambda t, m=0.0, k=1.0: Framed(rows, d, t, lead, gap).fill(normal(rows, d, m=m, k=k))  # noqa: E731
        self.rows, self.d, self.stream, self.block, self.lead, self.gap = rows, d, stream, block, lead, gap
        self.x, self.dx = frame(stream, mean, 1.5), frame(stream)
        self.dh = frame(block)
        self.f = frame(block, mean, 0.7) if join else None
        norm = lambda: ra.Norm(normal(d, m=1.0, k=0.2).to(param), normal(d, k=0.2).to(param) if bias else None, kind=kind, eps=1e-5)  # noqa: E731
        self.pre, self.post = norm(), norm() if join else None
        self.gate = None
        if join and gate == "vector":
            self.gate = normal(d, k=0.5).to(param)
        elif join and gate == "matrix":
            self.gate = frame(block).t
        self.alpha, self.beta = 0.875, 1.25

    def forward(self, out=None, h=None):
        f = None if self.f is None else self.f.t
        return ra.ra_norm_block(self.x.t, f, post=self.post, gate=self.gate, alpha=self.alpha, beta=self.beta, pre=self.pre, out=out, h=h,
                                dtype=None if f is not None or h is not None else self.block)

    def check_forward(self):
        x_out, h = Framed(self.rows, self.d, self.stream, self.lead, self.gap), Framed(self.rows, self.d, self.block, self.lead, self.gap)
        x, got, kept = self.forward(x_out.t if self.f is not None else None, h.t)
        if self.f is not None:
            want, size = join64(self.x.t, self.f.t, self.post, self.gate, self.alpha, self.beta)
            check(x, want, CHAIN * size + half_step(self.stream) * want.abs(), "x'")
            x_out.intact("x'")
        want, size, _, _, m, rstd = _norm64(x.double(), self.pre)  # of the row as it is stored
        check(got, want, CHAIN * size + half_step(self.block) * want.abs(), "h")
        h.intact("h")
        mean = x.double().abs().mean(1, keepdim=True)
        check(kept[:, 2:3], m, 70 * U * mean, "m")
        # d rstd = -rstd^3 / 2 d var, and var is off by 70 u of itself and by what m is off, squared
        check(kept[:, 3:4], rstd, 100 * U * rstd + rstd ** 3 * (70 * U * mean) ** 2, "rstd")
        if self.post is not None:
            _, _, _, _, m, rstd = _norm64(self.f.t.double(), self.post)
            mean = self.f.t.double().abs().mean(1, keepdim=True)
            check(kept[:, 0:1], m, 70 * U * mean, "m of f")
            check(kept[:, 1:2], rstd, 100 * U * rstd + rstd ** 3 * (70 * U * mean) ** 2, "rstd of f")
        return x, got, kept

    def check_backward(self, x, kept):
        f = None if self.f is None else self.f.t
        alpha, beta = self.alpha, self.beta
        want = grads64(self.dh.t, x, f, self.post, self.gate, alpha, beta, self.pre, self.dx.t)
        out = ra.NormBlockGrads()
        frames = {"dx": Framed(self.rows, self.d, self.stream, self.lead, self.gap)}
        if f is not None:
            frames["df"] = Framed(self.rows, self.d, self.block, self.lead, self.gap)
            if self.gate is not None and self.gate.dim() == 2:
                frames["gate"] = Framed(self.rows, self.d, self.block, self.lead, self.gap)
        for name in want:
            setattr(out, name, frames[name].t if name in frames else torch.full((self.d,), float("nan"), device="cuda"))
        args = dict(f=f, post=self.post, gate=self.gate, alpha=alpha, beta=beta, pre=self.pre, dx=self.dx.t)
        ra.ra_norm_block_grad(self.dh.t, x, kept, out=out, **args)
        for name, (w, size) in want.items():
            t = getattr(out, name)
            check(t, w, CHAIN * size + half_step(t.dtype) * w.abs(), name)
        for name, frame in frames.items():
            frame.intact(name)
        held = {name: getattr(out, name).clone() for name in want}
        ra.ra_norm_block_grad(self.dh.t, x, kept, out=out, **args)
        for name in want:
            assert torch.equal(getattr(out, name), held[name]), name  # the same bits again
        return out


@pytest.mark.parametrize("stream,block", TYPES)
@pytest.mark.parametrize("rows,d", SIZES)
def test_sizes(rows, d, stream, block):
    for k, (kind, gate) in enumerate((("layer", "vector"), ("rms", "matrix"), ("layer", None))):
        c = _Case(rows, d, stream, block, kind, gate, join=k < 2, bias=kind == "layer")
        x, _, kept = c.check_forward()
        c.check_backward(x, kept)


@pytest.mark.parametrize("stream,block", TYPES)
@pytest.mark.parametrize("d,lead,gap", [(64, 8, 8), (512, 1, 0), (1000, 0, 3), (2048, 3, 5), (4104, 2, 2), (9000, 1, 0)])
def test_layouts(d, lead, gap, stream, block):
    for kind, gate, param in (("rms", "vector", BF16), ("layer", "matrix", F32)):
        c = _Case(37, d, stream, block, kind, gate, lead=lead, gap=gap, param=param)
        x, _, kept = c.check_forward()
        c.check_backward(x, kept)


@pytest.mark.parametrize("stream,block", TYPES)
@pytest.mark.parametrize("rows,d", [(300, 4999), (200, 12000), (130, 11999), (70, 24000), (50, 27999), (40, 32760)])
def test_rows_shared_by_a_cluster(rows, d, stream, block):
    """Two to eight blocks a row, with several rows each, and columns that do not fill the last block's share."""
    for kind, gate in (("layer", "vector"), ("rms", "matrix")):
        c = _Case(rows, d, stream, block, kind, gate)
        x, _, kept = c.check_forward()
        c.check_backward(x, kept)


def test_parts_that_are_not_there():
    """No post norm, no gate, no gains, no pre norm, no gradient of one side."""
    rows, d = 50, 640
    for stream, block in TYPES:
        for post in (None, ra.Norm(kind="rms"), ra.Norm(bias=torch.ones(d, device="cuda"))):
            for gated in (False, True):
                c = _Case(rows, d, stream, block, "layer", "vector" if gated else None)
                c.post = post
                x, _, kept = c.check_forward()
                c.check_backward(x, kept)
                # without a norm ahead: the join alone
                x2, h, kept2 = ra.ra_norm_block(c.x.t, c.f.t, post=post, gate=c.gate, alpha=c.alpha, beta=c.beta)
                assert h is None and torch.equal(x2, x) and not bool(kept2[:, 2:].any())
                g = ra.ra_norm_block_grad(None, x2, kept2, f=c.f.t, post=post, gate=c.gate, alpha=c.alpha, beta=c.beta, dx=c.dx.t)
                want = grads64(None, x2, c.f.t, post, c.gate, c.alpha, c.beta, None, c.dx.t)
                for name in ("dx", "df"):
                    w, size = want[name]
                    check(getattr(g, name), w, CHAIN * size + half_step(getattr(g, name).dtype) * w.abs(), name)
                # without a gradient of the stream
                g = ra.ra_norm_block_grad(c.dh.t, x, kept, f=c.f.t, post=post, gate=c.gate, alpha=c.alpha, beta=c.beta, pre=c.pre)
                want = grads64(c.dh.t, x, c.f.t, post, c.gate, c.alpha, c.beta, c.pre, None)
                for name in ("dx", "df", "pre_gain", "pre_bias"):
                    w, size = want[name]
                    check(getattr(g, name), w, CHAIN * size + half_step(getattr(g, name).dtype) * w.abs(), name)
    x, h, kept = ra.ra_norm_block(c.x.t, pre=c.pre, keep=False, dtype=block)
    assert x is c.x.t and kept is None


def test_only_the_gradients_asked_for():
    c = _Case(40, 256, F32, F32, "layer", "vector")
    x, _, kept = c.forward()
    args = dict(f=c.f.t, post=c.post, gate=c.gate, alpha=c.alpha, beta=c.beta, pre=c.pre, dx=c.dx.t)
    whole = ra.ra_norm_block_grad(c.dh.t, x, kept, **args)
    for name in ra.NormBlockGrads.__slots__:
        out = ra.NormBlockGrads(**{name: torch.full_like(getattr(whole, name), 7.0)})
        ra.ra_norm_block_grad(c.dh.t, x, kept, out=out, **args)
        assert torch.equal(getattr(out, name), getattr(whole, name)), name
    d = c.d
    flat = torch.zeros(5 * d + 1, device="cuda")  # a worker's row: the vectors off 16-byte boundaries
    out = ra.NormBlockGrads(gate=flat[1:1 + d], post_gain=flat[1 + d:1 + 2 * d], post_bias=flat[1 + 2 * d:1 + 3 * d], pre_gain=flat[1 + 3 * d:1 + 4 * d],
                            pre_bias=flat[1 + 4 * d:])
    for k in (1, 2):
        ra.ra_norm_block_grad(c.dh.t, x, kept, out=out, accumulate=True, **args)
        for name in ("gate", "post_gain", "post_bias", "pre_gain", "pre_bias"):
            assert torch.equal(getattr(out, name), k * getattr(whole, name)), name
    assert float(flat[0]) == 0


def test_in_place():
    for d in (256, 257, 9000):
        c = _Case(21, d, F32, BF16, "layer", "vector")
        x, h, kept = c.forward()
        held = c.x.t.clone()
        got, h2, kept2 = ra.ra_norm_block(held, c.f.t, post=c.post, gate=c.gate, alpha=c.alpha, beta=c.beta, pre=c.pre, out=held)
        assert got is held and torch.equal(held, x) and torch.equal(h2, h) and torch.equal(kept, kept2)
        args = dict(f=c.f.t, post=c.post, gate=c.gate, alpha=c.alpha, beta=c.beta, pre=c.pre)
        want = ra.ra_norm_block_grad(c.dh.t, x, kept, dx=c.dx.t, **args).dx
        grad = c.dx.t.clone()
        ra.ra_norm_block_grad(c.dh.t, x, kept, dx=grad, out=ra.NormBlockGrads(dx=grad), **args)
        assert torch.equal(grad, want)


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("gate", ["vector", "matrix"])
def test_against_differences(kind, gate):
    """Every gradient against central differences of the 64-bit form, on values small enough that the differences' own error (the
    third derivative times h^2) stays far below what a wrong term would make."""
    rows, d, h = 3, 16, 1e-4
    c = _Case(rows, d, F32, F32, kind, gate)
    x, _, kept = c.forward()
    got = ra.ra_norm_block_grad(c.dh.t, x, kept, f=c.f.t, post=c.post, gate=c.gate, alpha=c.alpha, beta=c.beta, pre=c.pre, dx=c.dx.t)
    names = ["x", "f", "gate", "post_gain", "post_bias", "pre_gain", "pre_bias"]
    values = [t.double() for t in (c.x.t, c.f.t, c.gate, c.post.gain, c.post.bias, c.pre.gain, c.pre.bias)]

    def loss(v):
        x0, f, g, pg, pb, qg, qb = v
        x1, _ = join64(x0, f, ra.Norm(pg, pb, kind=kind), g, c.alpha, c.beta)
        return (c.dx.t.double() * x1).sum() + (c.dh.t.double() * _norm64(x1, ra.Norm(qg, qb, kind=kind))[0]).sum()

    for k, name in enumerate(names):
        mine = {"x": got.dx, "f": got.df}.get(name, getattr(got, name, None)).double()
        flat = values[k].reshape(-1)
        for i in range(0, flat.numel(), 5):
            diff = 0
            for sign in (1, -1):
                moved = flat.clone()
                moved[i] += sign * h
                diff = diff + sign * loss(values[:k] + [moved.view_as(values[k])] + values[k + 1:])
            diff = float(diff) / (2 * h)
            # covers the differences (h^2 = 1e-8 times derivatives below 1e3) and binary32's 512 u of magnitudes below 1e2
            assert abs(diff - float(mine.reshape(-1)[i])) < 4e-3 * (1 + abs(diff)), (name, i)


def test_non_finite_rows_stay_in_their_row():
    c = _Case(6, 128, F32, F32, "layer", "vector")
    c.f.t[2, 5] = float("nan")
    c.x.t[4, 7] = float("inf")
    x, h, kept = c.forward()
    ok = torch.tensor([0, 1, 3, 5], device="cuda")
    assert bool(torch.isnan(x[2]).all()) and bool(torch.isnan(h[2]).all()) and bool(torch.isnan(h[4]).all()) and float(x[4, 7]) == float("inf")
    assert bool(torch.isfinite(x[ok]).all()) and bool(torch.isfinite(h[ok]).all()) and bool(torch.isfinite(kept[ok]).all())


def test_a_large_mean_and_constant_rows():
    """The second moment is that of the differences from the mean: rows far from zero keep their variance."""
    rows, d = 8, 2048
    v = torch.randn(rows, d, generator=torch.Generator(device="cuda").manual_seed(5), device="cuda") + 1000.0
    v[3] = 7.0
    n = ra.Norm(kind="layer", eps=1e-5)
    _, h, kept = ra.ra_norm_block(v, pre=n, dtype=F32)
    want, _, _, _, m, rstd = _norm64(v.double(), n)
    # the mean is off by at most 70 u * 1000 = 0.0042, and so is each difference
    check(h, want, 0.0042 * rstd.clamp(max=2) + 1e-3 * want.abs(), "h")
    assert not bool(h[3].any()) and abs(float(kept[3, 3]) - 1e-5 ** -0.5) < 1e-2


def test_streams_and_graphs():
    c = _Case(100, 512, BF16, BF16, "layer", "vector")
    x, h, kept = c.forward()
    args = dict(f=c.f.t, post=c.post, gate=c.gate, alpha=c.alpha, beta=c.beta, pre=c.pre, dx=c.dx.t)
    want = ra.ra_norm_block_grad(c.dh.t, x, kept, **args)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    grads = [ra.ra_norm_block_grad(c.dh.t, x, kept, stream=s, **args) for s in streams]
    torch.cuda.synchronize()
    for g in grads:
        for name in ra.NormBlockGrads.__slots__:
            assert torch.equal(getattr(g, name), getattr(want, name))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x2, h2, kept2 = c.forward()
        g2 = ra.ra_norm_block_grad(c.dh.t, x2, kept2, **args)
    c.f.t.mul_(2)
    for _ in range(2):
        graph.replay()
    x, h, kept = c.forward()
    want = ra.ra_norm_block_grad(c.dh.t, x, kept, **args)
    assert torch.equal(x, x2) and torch.equal(h, h2)
    for name in ra.NormBlockGrads.__slots__:
        assert torch.equal(getattr(g2, name), getattr(want, name))


def test_empty_calls():
    e = torch.empty(0, 8, device="cuda")
    n = ra.Norm(torch.ones(8, device="cuda"))
    x, h, kept = ra.ra_norm_block(e, e, post=n, pre=n)
    g = ra.ra_norm_block_grad(h, x, kept, f=e, post=n, pre=n)
    assert h.shape == (0, 8) and g.dx.shape == (0, 8) and not bool(g.pre_gain.any()) and not bool(g.post_gain.any())
    g = ra.ra_norm_block_grad(h, x, kept, pre=n)
    assert not bool(g.pre_gain.any())
    held = ra.NormBlockGrads(pre_gain=torch.full((8,), 3.0, device="cuda"))
    ra.ra_norm_block_grad(h, x, kept, f=e, post=n, pre=n, out=held, accumulate=True)
    assert bool((held.pre_gain == 3).all())
    z = torch.empty(5, 0, device="cuda")
    assert ra.ra_norm_block(z, pre=ra.Norm(), dtype=F32)[1].shape == (5, 0)


def test_past_32_bit_offsets():
    rows, d = (1 << 20) + 5, 2056  # 2.16 G values
    x = torch.zeros(rows, d, dtype=BF16, device="cuda")
    at = torch.tensor([0, rows // 2, rows - 1], device="cuda")
    x[at] = torch.randn(3, d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).to(BF16)
    n = ra.Norm(torch.full((d,), 2.0, device="cuda"), kind="rms")
    _, h, kept = ra.ra_norm_block(x, pre=n)
    want, size = _norm64(x[at].double(), n)[:2]
    check(h[at], want, CHAIN * size + half_step(BF16) * want.abs())
    assert not bool(h[1:1000].any()) and not bool(h[-1000:-1].any())
    g = ra.ra_norm_block_grad(h, x, kept, pre=n, dx=h, out=ra.NormBlockGrads(dx=torch.empty_like(x)))
    want, size = grads64(h[at], x[at], None, None, None, 1, 1, n, h[at])["dx"]
    check(g.dx[at], want, CHAIN * size + half_step(BF16) * want.abs())
    del x, h, g
    torch.cuda.empty_cache()


def test_refusals():
    t, b = torch.zeros(4, 16, device="cuda"), torch.zeros(4, 16, dtype=BF16, device="cuda")
    n, kept = ra.Norm(torch.ones(16, device="cuda")), torch.zeros(4, 4, device="cuda")
    for call in (lambda: ra.ra_norm_block(t), lambda: ra.ra_norm_block(t, post=n, pre=n), lambda: ra.ra_norm_block(t, gate=t[0], pre=n),
                 lambda: ra.ra_norm_block(t, t[:2], pre=n), lambda: ra.ra_norm_block(t, t, gate=t[:2]), lambda: ra.ra_norm_block(t, t, h=t.clone()),
                 lambda: ra.ra_norm_block(t, pre=ra.Norm(torch.ones(8, device="cuda"))), lambda: ra.ra_norm_block(t, pre=n, out=t),
                 lambda: ra.ra_norm_block_grad(t, t, kept), lambda: ra.ra_norm_block_grad(None, t, kept), lambda: ra.ra_norm_block_grad(t, t, None, pre=n),
                 lambda: ra.ra_norm_block_grad(t, t, kept[:2], pre=n), lambda: ra.ra_norm_block_grad(t, t, kept, pre=n, accumulate=True),
                 lambda: ra.ra_norm_block_grad(t, t, kept, pre=n, out=ra.NormBlockGrads(df=t.clone())),
                 lambda: ra.ra_norm_block_grad(t, t, kept, pre=n, post=n)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: ra.ra_norm_block(b, t, pre=n), lambda: ra.ra_norm_block(b, pre=n, dtype=F32), lambda: ra.ra_norm_block(t, b, pre=n, h=t.clone()),
                 lambda: ra.ra_norm_block(t, t, pre="layer"), lambda: ra.ra_norm_block(t, t, gate=b), lambda: ra.ra_norm_block(t, t, out=b),
                 lambda: ra.ra_norm_block(t, pre=ra.Norm(t[0], b[0])), lambda: ra.ra_norm_block_grad(t, t, kept, pre=n, out=t),
                 lambda: ra.ra_norm_block_grad(t, t, kept, pre=n, out=ra.NormBlockGrads(pre_gain=b[0]))):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(ra.RaError, match="OVERLAP"):
        ra.ra_norm_block(t, t, pre=n, h=t)
    with pytest.raises(ra.RaError, match="INVALID"):
        ra.ra_norm_block_grad(t, t.clone(), kept, pre=n, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    wide = torch.zeros(2, 32776, device="cuda")
    with pytest.raises(ra.RaError, match="UNSUPPORTED"):
        ra.ra_norm_block(wide, pre=ra.Norm(), dtype=F32)
