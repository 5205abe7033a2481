"""ra_linear, ra_linear_dgrad and ra_linear_wgrad against plain forms in 64
bits, at the sizes, strides and values where they can go wrong."""
from __future__ import annotations

import pytest
import torch

import gradient_ring_all_gb300 as ra
from gradient_ring_all_gb300 import operators
from operator_reference import Framed, act64, check, pack64, rounding, slope64, sum_bound, values64

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
ACTS = ["none", "relu", "gelu", "silu"]

# (m, k, n): single elements, single tokens, tile edges and one past them, long and short sums, odd everything
SIZES = [(1, 1, 1), (1, 64, 8), (1, 2048, 512), (2, 8, 4000), (7, 16, 40), (33, 65, 31), (64, 64, 64), (127, 128, 129), (128, 72, 256),
         (129, 200, 257), (200, 1, 300), (3, 5000, 5), (256, 512, 128), (300, 1000, 520), (513, 333, 77), (1024, 96, 1032)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from gradient_ring_all_gb300 import build
    build.build()
    ra.load()


def _normal(seed, *shape, dtype=BF16, s=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * s).to(dtype)


def _framed(t, lead, gap):
    return Framed(t.shape[0], t.shape[1], t.dtype, lead, gap).fill(t)


def _forward64(x, w, bias, act, residual):
    """(z, y, the products' magnitudes)"""
    z = x.double() @ w.double()
    size = x.double().abs() @ w.double().abs()
    if bias is not None:
        z = z + bias.double()
        size = size + bias.double().abs()
    y = act64(z, act)
    if residual is not None:
        y = y + residual.double()
    return z, y, size


def _forward_bound(k, z, y, size, dtype, residual):
    extra = 0 if residual is None else residual.double().abs()
    return 1.13 * sum_bound(k + 1) * size + 2.0 ** -20 * z.abs() + rounding(dtype) * (y.abs() + 2.0 ** -12 * extra) + 2.0 ** -23 * extra


@pytest.mark.parametrize("out_type", [BF16, F32])
@pytest.mark.parametrize("m,k,n", SIZES)
def test_forward_by_size(m, k, n, out_type):
    x, w = _normal(m, m, k), _normal(n, k, n, s=k ** -0.5)
    bias, residual = _normal(3, n, dtype=F32), _normal(4, m, n)
    out = Framed(m, n, out_type)
    ra.ra_linear(x, w, bias=bias, act="gelu", residual=residual, out=out.t)
    z, y, size = _forward64(x, w, bias, "gelu", residual)
    check(out.t, y, _forward_bound(k, z, y, size, out_type, residual))
    out.intact("linear")
    again = ra.ra_linear(x, w, bias=bias, act="gelu", residual=residual, dtype=out_type)
    assert torch.equal(again, out.t)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("bias_type", [None, F32, BF16])
@pytest.mark.parametrize("res_type", [None, F32, BF16])
@pytest.mark.parametrize("out_type", [BF16, F32])
def test_forward_by_epilogue(act, bias_type, res_type, out_type):
    for m, k, n in ((70, 96, 136), (5, 40, 67)):
        x, w = _normal(1, m, k), _normal(2, k, n, s=k ** -0.5 * 3)
        bias = None if bias_type is None else _normal(3, n, dtype=bias_type)
        residual = None if res_type is None else _normal(4, m, n, dtype=res_type)
        got = ra.ra_linear(x, w, bias=bias, act=act, residual=residual, dtype=out_type)
        z, y, size = _forward64(x, w, bias, act, residual)
        check(got, y, _forward_bound(k, z, y, size, out_type, residual))


@pytest.mark.parametrize("lx,gx,lw,gw,ly,gy", [(8, 8, 16, 8, 8, 0), (0, 1, 0, 0, 0, 0), (1, 0, 0, 1, 1, 1), (0, 0, 3, 0, 0, 3), (4, 4, 4, 4, 2, 2)])
def test_forward_by_strides(lx, gx, lw, gw, ly, gy):
    m, k, n = 140, 104, 72
    x, w, r = _framed(_normal(1, m, k), lx, gx), _framed(_normal(2, k, n), lw, gw), _framed(_normal(3, m, n), ly, gy)
    out = Framed(m, n, BF16, ly, gy)
    ra.ra_linear(x.t, w.t, residual=r.t, out=out.t)
    z, y, size = _forward64(x.t, w.t, None, "none", r.t)
    check(out.t, y, _forward_bound(k, z, y, size, BF16, r.t))
    out.intact("linear")
    ra.ra_linear(x.t, w.t, residual=r.t, out=r.t)  # in place on the residual
    assert torch.equal(r.t, out.t)
    r.intact("linear in place")


@pytest.mark.parametrize("m,k,n", [(1, 64, 32), (5, 40, 67), (130, 136, 256), (257, 200, 1000), (64, 2048, 96)])
@pytest.mark.parametrize("act", ["none", "gelu"])
def test_forward_keeps_the_preactivation(m, k, n, act):
    x, w, bias = _normal(1, m, k), _normal(2, k, n, s=k ** -0.5), _normal(3, n, dtype=F32)
    groups = -(-n // 32)
    fq, fe = Framed(m, groups * 32, torch.int8), Framed(m, groups, torch.uint8)
    kept = ra.Checkpoint8(m, n, q=fq.t, e=fe.t)
    y = ra.ra_linear(x, w, bias=bias, act=act, save=kept)
    z, want, size = _forward64(x, w, bias, act, None)
    check(y, want, _forward_bound(k, z, want, size, BF16, None))
    fq.intact("save")
    fe.intact("save")
    assert torch.equal(y, ra.ra_linear(x, w, bias=bias, act=act))
    # half a step, at most 1/127.5 of the group's largest magnitude, with z itself off by its bound
    off = sum_bound(k + 1) * size
    top = torch.nn.functional.pad(z.abs() + off, (0, groups * 32 - n)).view(m, groups, 32).amax(2).repeat_interleave(32, 1)[:, :n]
    check(ra.ra_checkpoint8_unpack(kept, dtype=F32), z, top / 127.5 * (1 + 2.0 ** -20) + off)
    assert not bool(kept.q[:, n:].any())
    # and where z is exact (small whole numbers), the bytes are the definition's
    xi, wi = torch.randint(-2, 3, (m, k), device="cuda").to(BF16), torch.randint(-2, 3, (k, n), device="cuda").to(BF16)
    ra.ra_linear(xi, wi, act=act, save=kept)
    q, e = pack64((xi.double() @ wi.double()))
    assert torch.equal(kept.q, q) and torch.equal(kept.e, e)


@pytest.mark.parametrize("m,k,n", SIZES)
@pytest.mark.parametrize("act", ["none", "silu"])
def test_dgrad_by_size(m, k, n, act):
    dy, w = _normal(m, m, n), _normal(n, k, n, s=n ** -0.5)
    kept = ra.ra_checkpoint8_pack(_normal(5, m, k, s=2.0)) if act != "none" else None
    for out_type in (BF16, F32):
        out = Framed(m, k, out_type)
        ra.ra_linear_dgrad(dy, w, saved=kept, act=act, out=out.t)
        z = values64(kept.q, kept.e, k) if kept else torch.zeros(m, k, dtype=torch.float64, device="cuda")
        g, size = dy.double() @ w.double().t(), dy.double().abs() @ w.double().t().abs()
        want = g * slope64(z, act)
        check(out.t, want, 1.13 * sum_bound(n) * size + 2.0 ** -20 * g.abs() * (1 + z.abs()) + rounding(out_type) * want.abs())
        out.intact("dgrad")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("res_type", [None, F32, BF16])
@pytest.mark.parametrize("lead,gap", [(0, 0), (8, 8), (1, 2)])
def test_dgrad_by_epilogue(act, res_type, lead, gap):
    m, k, n = 150, 100, 72
    dy, w = _framed(_normal(1, m, n), lead, gap), _framed(_normal(2, k, n), lead, gap)
    kept = ra.ra_checkpoint8_pack(_normal(5, m, k, s=2.0))
    residual = None if res_type is None else _framed(_normal(4, m, k, dtype=res_type), lead, gap)
    out = Framed(m, k, BF16, lead, gap)
    ra.ra_linear_dgrad(dy.t, w.t, saved=kept, act=act, residual=None if residual is None else residual.t, out=out.t)
    z = values64(kept.q, kept.e, k)
    g, size = dy.t.double() @ w.t.double().t(), dy.t.double().abs() @ w.t.double().t().abs()
    want = g * slope64(z, act)
    extra = 0 if residual is None else residual.t.double()
    want = want + extra
    bound = 1.13 * sum_bound(n) * size + 2.0 ** -20 * g.abs() * (1 + z.abs()) + rounding(BF16) * want.abs()
    check(out.t, want, bound + (0 if residual is None else 2.0 ** -22 * extra.abs()))
    out.intact("dgrad")


@pytest.mark.parametrize("m,k,n", SIZES)
@pytest.mark.parametrize("out_type", [BF16, F32])
def test_wgrad_by_size(m, k, n, out_type):
    x, dy = _normal(m, m, k), _normal(n, m, n)
    out = Framed(k, n, out_type)
    db = torch.full((n + 2,), 7.0, device="cuda")
    ra.ra_linear_wgrad(x, dy, out=out.t, bias_grad=db[1:n + 1])
    want, size = x.double().t() @ dy.double(), x.double().t().abs() @ dy.double().abs()
    check(out.t, want, sum_bound(m) * size + rounding(out_type) * want.abs())
    out.intact("wgrad")
    check(db[1:n + 1], dy.double().sum(0), sum_bound(m) * dy.double().abs().sum(0))
    assert float(db[0]) == 7 and float(db[n + 1]) == 7
    again, db2 = ra.ra_linear_wgrad(x, dy, dtype=out_type, bias_grad=True)
    assert torch.equal(again, out.t) and torch.equal(db2, db[1:n + 1])


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m,k,n", [(1, 32, 8), (65, 100, 40), (300, 257, 129), (700, 64, 512)])
def test_wgrad_from_a_checkpoint(act, m, k, n):
    kept = ra.ra_checkpoint8_pack(_normal(5, m, k, s=2.0))
    dy = _normal(1, m, n)
    z = values64(kept.q, kept.e, k)
    a = act64(z, act)
    want, size = a.t() @ dy.double(), a.t().abs() @ dy.double().abs()
    # without an activation the checkpoint's values are exact bf16 operands; else act(z) is rounded to bf16 once
    operand = 0.0 if act == "none" else 2.0 ** -8
    for out_type in (F32, BF16):
        dw, db = ra.ra_linear_wgrad(kept, dy, act=act, dtype=out_type, bias_grad=True)
        own = operand * size + (0 if act == "none" else 2.0 ** -20 * (z.abs().t() @ dy.double().abs()))
        check(dw, want, own + sum_bound(m) * size * (1 + operand) + rounding(out_type) * want.abs())
        check(db, dy.double().sum(0), sum_bound(m) * dy.double().abs().sum(0))


@pytest.mark.parametrize("out_type", [BF16, F32])
@pytest.mark.parametrize("lead,gap", [(0, 0), (8, 8), (1, 2)])
def test_wgrad_accumulates_over_micro_batches(out_type, lead, gap):
    m, k, n = 96, 80, 48
    dw, db = Framed(k, n, out_type, lead, gap), torch.zeros(n, device="cuda")
    dw.t.zero_()
    want = torch.zeros(k, n, dtype=torch.float64, device="cuda")
    bound, b64 = 0, 0
    for step in range(3):
        x, dy = _framed(_normal(step, m, k), lead, gap), _framed(_normal(step + 9, m, n), lead, gap)
        ra.ra_linear_wgrad(x.t, dy.t, out=dw.t, bias_grad=db, accumulate=True)
        want = want + x.t.double().t() @ dy.t.double()
        bound = bound + sum_bound(m + 1) * (x.t.double().t().abs() @ dy.t.double().abs()) + rounding(out_type) * want.abs()
        b64 = b64 + dy.t.double().sum(0)
    check(dw.t, want, 1.01 * bound + 6 * rounding(out_type) * bound)
    check(db, b64, sum_bound(3 * m) * 3 * m * 4)
    dw.intact("wgrad accumulate")


@pytest.mark.parametrize("out_type", [BF16, F32])
def test_last_tiles_made_in_parts(out_type):
    """Sizes whose last wave of tiles is split along k, ragged ones, in all three products; and the same without the room."""
    lib = operators._load()
    m, k, n = 2500, 4100, 2200
    x, w = _normal(1, m, 4104)[:, :k], _normal(2, k, n, s=k ** -0.5)
    bias, residual = _normal(3, n, dtype=F32), _normal(4, m, n)
    assert lib.ra_linear_split_bytes(m, n, k) > 0
    kept, out = ra.Checkpoint8(m, n), Framed(m, n, out_type, 0, 16)
    ra.ra_linear(x, w, bias=bias, act="gelu", residual=residual, save=kept, out=out.t)
    z, y, size = _forward64(x, w, bias, "gelu", residual)
    bound = _forward_bound(k, z, y, size, out_type, residual)
    check(out.t, y, bound)
    out.intact("split")
    groups = -(-n // 32)
    off = sum_bound(k + 1) * size
    top = torch.nn.functional.pad(z.abs() + off, (0, groups * 32 - n)).view(m, groups, 32).amax(2).repeat_interleave(32, 1)[:, :n]
    check(ra.ra_checkpoint8_unpack(kept, dtype=F32), z, top / 127.5 * (1 + 2.0 ** -20) + off)
    again = ra.ra_linear(x, w, bias=bias, act="gelu", residual=residual, dtype=out_type)
    assert torch.equal(again, out.t)
    small = torch.empty(256, dtype=torch.uint8, device="cuda")
    check(ra.ra_linear(x, w, bias=bias, act="gelu", residual=residual, dtype=out_type, workspace=small), y, bound)
    # x of the forward product as dy of the others: rows of dx, and of dw, over 4100
    assert lib.ra_linear_split_bytes(m, n, k) > 0 and lib.ra_linear_split_bytes(n, m, k) > 0
    wt = _normal(5, n, k, s=k ** -0.5)
    z8 = ra.ra_checkpoint8_pack(_normal(6, m, n, s=2.0))
    got = ra.ra_linear_dgrad(x, wt, saved=z8, act="silu", dtype=out_type)
    zz = values64(z8.q, z8.e, n)
    g, gsize = x.double() @ wt.double().t(), x.double().abs() @ wt.double().t().abs()
    want = g * slope64(zz, "silu")
    check(got, want, 1.13 * sum_bound(k) * gsize + 2.0 ** -20 * g.abs() * (1 + zz.abs()) + rounding(out_type) * want.abs())
    a, dy = _normal(7, k, n), _normal(8, k, m + 4)[:, :m]
    dw, db = ra.ra_linear_wgrad(a, dy, dtype=out_type, bias_grad=True)
    want, size = a.double().t() @ dy.double(), a.double().t().abs() @ dy.double().abs()
    check(dw, want, sum_bound(k) * size + rounding(out_type) * want.abs())
    check(db, dy.double().sum(0), sum_bound(k) * dy.double().abs().sum(0))


@pytest.mark.parametrize("out_type", [BF16, F32])
@pytest.mark.parametrize("m,k,n", [(300, 4104, 328), (129, 4096, 1000), (257, 3210, 2081), (700, 5000, 96)])
def test_pairs_that_split_k(m, k, n, out_type):
    """Long sums into few tiles, two and four ways, in all three products: with every part of the epilogue."""
    x, w = _normal(1, m, k), _normal(2, k, n, s=k ** -0.5)
    bias, residual = _normal(3, n, dtype=F32), _normal(4, m, n)
    kept, out = ra.Checkpoint8(m, n), Framed(m, n, out_type, 0, 8)
    ra.ra_linear(x, w, bias=bias, act="gelu", residual=residual, save=kept, out=out.t)
    z, y, size = _forward64(x, w, bias, "gelu", residual)
    check(out.t, y, _forward_bound(k, z, y, size, out_type, residual))
    out.intact("pairs split")
    groups = -(-n // 32)
    off = sum_bound(k + 1) * size
    top = torch.nn.functional.pad(z.abs() + off, (0, groups * 32 - n)).view(m, groups, 32).amax(2).repeat_interleave(32, 1)[:, :n]
    check(ra.ra_checkpoint8_unpack(kept, dtype=F32), z, top / 127.5 * (1 + 2.0 ** -20) + off)
    assert torch.equal(ra.ra_linear(x, w, bias=bias, act="gelu", residual=residual, dtype=out_type), out.t)
    wt = _normal(5, n, k, s=k ** -0.5)
    z8 = ra.ra_checkpoint8_pack(_normal(6, m, n, s=2.0))
    got = ra.ra_linear_dgrad(x, wt, saved=z8, act="silu", dtype=out_type)
    zz = values64(z8.q, z8.e, n)
    g, gsize = x.double() @ wt.double().t(), x.double().abs() @ wt.double().t().abs()
    want = g * slope64(zz, "silu")
    check(got, want, 1.13 * sum_bound(k) * gsize + 2.0 ** -20 * g.abs() * (1 + zz.abs()) + rounding(out_type) * want.abs())
    a, dy = _normal(7, k, m), _normal(8, k, n)
    dw, db = ra.ra_linear_wgrad(a, dy, dtype=out_type, bias_grad=True)
    want, size = a.double().t() @ dy.double(), a.double().t().abs() @ dy.double().abs()
    check(dw, want, sum_bound(k) * size + rounding(out_type) * want.abs())
    check(db, dy.double().sum(0), sum_bound(k) * dy.double().abs().sum(0))


@pytest.mark.parametrize("m", [1, 2, 3, 4, 5, 8, 9, 15, 16])
@pytest.mark.parametrize("k", [512, 1100, 4096])
def test_few_rows_split_k(m, k):
    """Every share of up to 16 rows among two, four and eight splits, whole and ragged columns."""
    for n in (64, 200, 2081):
        x, w = _normal(m, m, k), _normal(n, k, n, s=k ** -0.5)
        bias, residual = _normal(3, n), _normal(4, m, n, dtype=F32)
        kept = ra.Checkpoint8(m, n)
        for out_type in (BF16, F32):
            out = Framed(m, n, out_type)
            ra.ra_linear(x, w, bias=bias, act="silu", residual=residual, save=kept, out=out.t)
            z, y, size = _forward64(x, w, bias, "silu", residual)
            check(out.t, y, _forward_bound(k, z, y, size, out_type, residual))
            out.intact("few rows")
            groups = -(-n // 32)
            off = sum_bound(k + 1) * size
            top = torch.nn.functional.pad(z.abs() + off, (0, groups * 32 - n)).view(m, groups, 32).amax(2).repeat_interleave(32, 1)[:, :n]
            check(ra.ra_checkpoint8_unpack(kept, dtype=F32), z, top / 127.5 * (1 + 2.0 ** -20) + off)


@pytest.mark.parametrize("out_type", [BF16, F32])
@pytest.mark.parametrize("k", [511, 512, 513, 2047, 2048, 4100, 16384, 16390])
def test_a_single_token(k, out_type):
    """The form for one row: rounds of k whole, cut short and more than it takes, and weights of every alignment."""
    for n, lead, gap in ((1, 0, 0), (8, 0, 8), (67, 0, 0), (640, 8, 24), (1001, 1, 0)):
        x, w = _framed(_normal(1, 1, k), lead, 0), _framed(_normal(n, k, n, s=k ** -0.5), lead, gap)
        bias, residual = _normal(3, n, dtype=F32), _normal(4, 1, n)
        kept, out = ra.Checkpoint8(1, n), Framed(1, n, out_type, lead, gap)
        ra.ra_linear(x.t, w.t, bias=bias, act="gelu", residual=residual, save=kept, out=out.t)
        z, y, size = _forward64(x.t, w.t, bias, "gelu", residual)
        check(out.t, y, _forward_bound(k, z, y, size, out_type, residual))
        out.intact("token")
        groups = -(-n // 32)
        off = sum_bound(k + 1) * size
        top = torch.nn.functional.pad(z.abs() + off, (0, groups * 32 - n)).view(1, groups, 32).amax(2).repeat_interleave(32, 1)[:, :n]
        check(ra.ra_checkpoint8_unpack(kept, dtype=F32), z, top / 127.5 * (1 + 2.0 ** -20) + off)
        again = Framed(1, n, out_type, lead, gap)
        ra.ra_linear(x.t, w.t, bias=bias, act="gelu", residual=residual, out=again.t)
        assert torch.equal(again.t, out.t)


def test_a_single_token_with_values_that_are_not_finite():
    """An infinite or NaN weight reaches its own column alone, a value of x all of them."""
    k, n = 2048, 200
    x, w = _normal(1, 1, k), _normal(2, k, n)
    clean = ra.ra_linear(x, w, dtype=F32)
    w[700, 33], w[2047, 199], w[0, 0] = float("inf"), float("nan"), float("-inf")
    got = ra.ra_linear(x, w, dtype=F32)
    hit = torch.zeros(n, dtype=torch.bool, device="cuda")
    hit[[0, 33, 199]] = True
    assert torch.equal(got[0, ~hit], clean[0, ~hit]) and not bool(got[0, hit].isfinite().any())
    x[0, 5] = float("nan")
    assert bool(ra.ra_linear(x, w, dtype=F32).isnan().all())


@pytest.mark.parametrize("lead,gap", [(0, 0), (8, 0), (0, 8), (16, 8), (24, 24), (4, 4)])
@pytest.mark.parametrize("n", [8, 40, 56, 328, 1000])
def test_rows_on_16_byte_boundaries(lead, gap, n):
    """Results whose rows start on 16-byte but not on 32-byte boundaries, with columns up to any multiple of 8."""
    for m, k in ((37, 72), (300, 200), (16, 1024)):
        x, w, bias = _normal(1, m, k), _normal(2, k, n, s=k ** -0.5), _normal(3, n, dtype=F32)
        out = Framed(m, n, BF16, lead, gap)
        ra.ra_linear(x, w, bias=bias, act="relu", out=out.t)
        z, y, size = _forward64(x, w, bias, "relu", None)
        check(out.t, y, _forward_bound(k, z, y, size, BF16, None))
        out.intact("16-byte rows")


def test_past_32_bit_offsets():
    """An output of more than 2^31 values, beside inputs whose last rows start beyond 2^31 bytes."""
    m, k, n = 70_000, 64, 32_000
    x, w = _normal(1, m, k), _normal(2, k, n)
    y = ra.ra_linear(x, w)
    kept = ra.ra_checkpoint8_pack(y)
    for rows in ([0, 1, 255, 256], [m // 2, m // 2 + 1], [67_107, 67_108, 67_109], [m - 257, m - 2, m - 1]):
        z = x[rows].double() @ w.double()
        size = x[rows].double().abs() @ w.double().abs()
        check(y[rows], z, sum_bound(k) * size + rounding(BF16) * z.abs())
        q, e = pack64(y[rows])
        assert torch.equal(kept.q[rows], q) and torch.equal(kept.e[rows], e)
    back = ra.ra_checkpoint8_unpack(kept)
    assert torch.equal(back[-3:].double(), values64(kept.q[-3:], kept.e[-3:], n))
    dw = ra.ra_linear_wgrad(x, y, dtype=F32)
    cols = [0, 1, n // 2, n - 1]
    want, size = x.double().t() @ y[:, cols].double(), x.double().t().abs() @ y[:, cols].double().abs()
    check(dw[:, cols], want, sum_bound(m) * size + rounding(F32) * want.abs())
    dx = ra.ra_linear_dgrad(y, w)
    rows = [0, 67_108, m - 1]
    want, size = y[rows].double() @ w.double().t(), y[rows].double().abs() @ w.double().t().abs()
    check(dx[rows], want, sum_bound(n) * size + rounding(BF16) * want.abs())


def test_empty_sums_and_nothing_to_do():
    e = lambda *s: torch.empty(*s, dtype=BF16, device="cuda")  # noqa: E731
    bias, res = _normal(1, 40, dtype=F32), _normal(2, 6, 40)
    y = ra.ra_linear(e(6, 0), e(0, 40), bias=bias, act="relu", residual=res, dtype=F32)
    check(y, act64(bias.double().expand(6, 40), "relu") + res.double(), 2.0 ** -22 * (bias.double().abs() + res.double().abs()))
    assert ra.ra_linear(e(0, 8), e(8, 40)).shape == (0, 40) and ra.ra_linear(e(6, 8), e(8, 0)).shape == (6, 0)
    assert not bool(ra.ra_linear_dgrad(e(6, 0), e(40, 0)).any())
    dw, db = ra.ra_linear_wgrad(e(0, 24), e(0, 40), bias_grad=True)
    assert dw.shape == (24, 40) and not bool(dw.any()) and not bool(db.any())
    held = torch.full((24, 40), 2.0, device="cuda")
    ra.ra_linear_wgrad(e(0, 24), e(0, 40), out=held, accumulate=True)
    assert bool((held == 2).all())


def test_non_finite_values_stay_in_their_rows():
    m, k, n = 200, 136, 264
    x, w = _normal(1, m, k), _normal(2, k, n)
    x[17, 5] = float("nan")
    x[130, 0] = float("inf")
    kept = ra.Checkpoint8(m, n)
    y = ra.ra_linear(x, w, act="relu", save=kept).double()
    rows = torch.zeros(m, dtype=torch.bool, device="cuda")
    rows[[17, 130]] = True
    assert bool(torch.isfinite(y[~rows]).all()) and bool(torch.isnan(y[17]).all())
    # +-inf by the sign of w's row, and relu's
    assert torch.equal(y[130], torch.where(w[0].double() > 0, float("inf"), 0.0).double())
    back = ra.ra_checkpoint8_unpack(kept, dtype=F32)
    assert bool(torch.isnan(back[rows]).all()) and bool(torch.isfinite(back[~rows]).all())
    # masked rows of zeros give zero gradients, and their NaN input none either where the product skips nothing
    dy = _normal(3, m, n)
    dy[50:60] = 0
    assert not bool(ra.ra_linear_dgrad(dy, w)[50:60].any())


@pytest.mark.parametrize("act", ["gelu", "silu"])
def test_gradients_against_differences(act):
    """dgrad and wgrad of y = act(z) W: central differences in 64 bits of L = sum(dy * y)."""
    m, k, n, h = 3, 32, 8, 1e-5
    kept = ra.ra_checkpoint8_pack(_normal(1, m, k, s=2.0))
    z = values64(kept.q, kept.e, k)
    w, dy = _normal(2, k, n), _normal(3, m, n)

    def loss(z, w):
        return float((dy.double() * (act64(z, act) @ w)).sum())

    dz = ra.ra_linear_dgrad(dy, w, saved=kept, act=act, dtype=F32).double()
    dw = ra.ra_linear_wgrad(kept, dy, act=act, dtype=F32).double()
    w64 = w.double()
    size = (dy.double().abs() @ w64.t().abs()).max().item()
    wsize = (act64(z, act).t().abs() @ dy.double().abs()).max().item()
    for i in range(0, m):
        for j in range(0, k, 5):
            d = torch.zeros_like(z)
            d[i, j] = h
            diff = (loss(z + d, w64) - loss(z - d, w64)) / (2 * h)
            # the differences' own error: h^2 times a third derivative below 1, and the loss's rounding over h
            assert abs(float(dz[i, j]) - diff) <= (1e-9 + 1e-9) * size + 1.13 * sum_bound(n) * size + 2.0 ** -18 * size
    for i in range(0, k, 7):
        for j in range(n):
            d = torch.zeros_like(w64)
            d[i, j] = h
            diff = (loss(z, w64 + d) - loss(z, w64 - d)) / (2 * h)
            assert abs(float(dw[i, j]) - diff) <= 1e-8 * wsize + (2.0 ** -8 + sum_bound(m)) * wsize


def test_streams_and_graphs():
    m, k, n = 160, 200, 136
    x, w = _normal(1, m, k), _normal(2, k, n + 1)[:, :n]  # w's rows are not 16-byte multiples apart: a workspace is used
    kept = ra.ra_checkpoint8_pack(_normal(3, m, k))
    dy = _normal(4, m, n)
    ids = torch.arange(m, device="cuda") % 50

    def work(stream=None):
        y = ra.ra_linear(x, w, act="silu", stream=stream)
        dz = ra.ra_linear_dgrad(dy, w, saved=kept, act="silu", stream=stream)
        dw, db = ra.ra_linear_wgrad(kept, dy, act="silu", bias_grad=True, stream=stream)
        de = ra.ra_embedding_grad(dz, ids, 50, stream=stream)
        back = ra.ra_checkpoint8_unpack(ra.ra_checkpoint8_pack(y, stream=stream), stream=stream)
        return [y, dz, dw, db, de, back, ra.ra_embedding_lookup(de, ids, stream=stream)]

    want = [t.clone() for t in work()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for given in (side, side.cuda_stream):
        got = work(given)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    with torch.cuda.stream(side):
        got = work()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = work()
    for t in got:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_refusals():
    x, w = _normal(1, 16, 24), _normal(2, 24, 32)
    dy, kept = _normal(3, 16, 32), ra.ra_checkpoint8_pack(_normal(4, 16, 24))
    with pytest.raises(TypeError):
        ra.ra_linear(x.float(), w)
    with pytest.raises(ValueError):
        ra.ra_linear(x, w[:20])
    with pytest.raises(ValueError):
        ra.ra_linear(x.t(), w)
    with pytest.raises(ValueError):
        ra.ra_linear(x, w, bias=torch.zeros(31, device="cuda"))
    with pytest.raises(ValueError):
        ra.ra_linear(x, w, act="tanh")
    with pytest.raises(ValueError):
        ra.ra_linear(x, w, save=ra.Checkpoint8(16, 24))
    with pytest.raises(ValueError):
        ra.ra_linear(x, w, residual=torch.zeros(16, 31, device="cuda"))
    with pytest.raises(TypeError):
        ra.ra_linear(x, w, dtype=torch.float16, out=torch.zeros(16, 32, device="cuda"))
    with pytest.raises(ra.RaError, match="OVERLAP"):
        sq = _normal(1, 24, 24)
        ra.ra_linear(x, sq, out=x)
    with pytest.raises(ra.RaError, match="OVERLAP"):
        big = torch.zeros(17 * 32, dtype=BF16, device="cuda")
        ra.ra_linear(x, w, residual=big[:512].view(16, 32), out=big[32:].view(16, 32))
    with pytest.raises(ValueError):
        ra.ra_linear_dgrad(dy, w, act="gelu")
    with pytest.raises(ValueError):
        ra.ra_linear_dgrad(dy, w, saved=ra.Checkpoint8(16, 32), act="gelu")
    with pytest.raises(ValueError):
        ra.ra_linear_wgrad(x, dy, act="gelu")
    with pytest.raises(ValueError):
        ra.ra_linear_wgrad(x, dy, accumulate=True)
    with pytest.raises(ValueError):
        ra.ra_linear_wgrad(kept, dy[:8])
    with pytest.raises(ValueError):
        ra.ra_linear_wgrad(x, dy, bias_grad=torch.zeros(32, dtype=BF16, device="cuda"))
    # column slices of one array may interleave: an output beside its input is no overlap
    both = torch.zeros(16, 56, dtype=BF16, device="cuda")
    both[:, :24] = x
    ra.ra_linear(both[:, :24], w, out=both[:, 24:])
    assert torch.equal(both[:, 24:], ra.ra_linear(x, w))
