"""ra_logprobs and ra_logprobs_grad against plain forms in 64 bits.

The bounds.  u = 2^-24, z = scale * logit, m a row's largest z.  An exponential
is off by 2^-21 of itself (the hardware's 2^x, 2 units) and by 4 u of its
argument's magnitude |z - m|; a sum passes a value through at most 350 additions
and rescalings at these sizes.  So log s is off by at most 400 u + 8 u + 4 u
times the mean of |z - m| under p, which is log s + entropy.  lse adds 2 u of
|m| and of itself; a log probability 4 u of |z - m|; the entropy, whose second
sum holds the terms times |z - m|, (400 + 4 |z - m|) u of each."""
from __future__ import annotations

import math

import pytest
import torch

import gradient_ring_all_gb300 as ra
from block_reference import U, alternatives64, distribution64, half_step
from operator_reference import Framed, check

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from gradient_ring_all_gb300 import build
    build.build()
    ra.load()


def _logits(rows, vocab, dtype, seed=0, s=2.5, lead=0, gap=0):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + rows * 31 + vocab)
    return Framed(rows, vocab, dtype, lead, gap).fill(torch.randn(rows, vocab, generator=g, device="cuda") * s)


def _ids(rows, vocab, seed=1, dtype=torch.int64):
    g = torch.Generator(device="cuda").manual_seed(seed)
    ids = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    ids[::5] = torch.tensor([-1, vocab, -100], device="cuda")[torch.arange(len(ids[::5]), device="cuda") % 3]
    return ids.to(dtype)


def _finite(v):
    return torch.where(torch.isfinite(v), v, 0.0)


def _bounds(z, m, log_s, h, p):
    """(of log s, of lse, of the entropy)"""
    base = (408 + 8 * _finite(log_s + h).clamp(min=0)) * U
    d = _finite(z - m.unsqueeze(1)).abs()
    return base, base + 4 * U * (_finite(m).abs() + _finite(m + log_s).abs()), base + ((410 + 8 * d) * p * d).nan_to_num().sum(1) * U


def _check(logits, ids, scale, top):
    rows, vocab = logits.shape
    r = ra.ra_logprobs(logits, ids, scale=scale, entropy=True, top=top)
    z, m, log_s, h, p = distribution64(logits, float(torch.tensor(scale, dtype=F32)))
    base, lse_bound, h_bound = _bounds(z, m, log_s, h, p)
    check(r.lse, m + log_s, lse_bound, "lse")
    check(r.entropy, h, h_bound + 2 * U * h.abs(), "entropy")
    assert not bool((r.entropy < 0).any())
    inside = (ids >= 0) & (ids < vocab)
    none = log_s == -INF
    if vocab:
        d = z.gather(1, ids.long().clamp(0, vocab - 1).unsqueeze(1)).squeeze(1) - m
        want = torch.where(none, -INF, d - log_s)
        check(r.logp, torch.where(inside, want, 0.0), base + 8 * U * (_finite(d).abs() + _finite(want).abs()), "logp")
    else:
        assert not bool(r.logp.any())
    if top:
        ids = alternatives64(logits, top).cuda()
        assert torch.equal(r.top_ids, ids)
        d = z.gather(1, ids.clamp(min=0)) - m.unsqueeze(1) if vocab else torch.zeros(rows, top, device="cuda", dtype=torch.float64)
        want = torch.where(ids < 0, -INF, d - log_s.unsqueeze(1))
        check(r.top_logp, want, base.unsqueeze(1) + 8 * U * (_finite(d).abs() + _finite(want).abs()), "top")
    else:
        assert r.top_ids is None and r.top_logp is None
    return r


SIZES = [(1, 1), (5, 2), (3, 7), (40, 31), (1, 32), (9, 33), (130, 257), (17, 1000), (20, 1024), (20, 1025), (6, 4097), (3, 16384), (4, 16385), (7, 32000),
         (2, 32001), (3, 32768), (2, 50001), (1, 131071), (19, 70000), (1, 262144), (2, 300001)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,vocab", SIZES)
def test_sizes(rows, vocab, dtype):
    z = _logits(rows, vocab, dtype)
    ids = _ids(rows, vocab)
    for scale, top in ((1.0, 0), (0.7, 1), (1.3, 8), (1.0, 32)):
        _check(z.t, ids, scale, top)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("lead,gap", [(1, 0), (0, 1), (3, 4), (8, 8)])
def test_layouts(lead, gap, dtype):
    for rows, vocab in ((50, 300), (5, 5000), (6, 33000)):
        z = _logits(rows, vocab, dtype, lead=lead, gap=gap)
        _check(z.t, _ids(rows, vocab, dtype=torch.int32), 0.9, 5)
        z.intact("logits")


@pytest.mark.parametrize("vocab", [300, 5003, 32000, 70001])
def test_rows_with_equal_and_ordered_logits(vocab):
    """Ties go to the lowest index; rising, falling and constant rows; a run of ties across the edge of what is taken."""
    n = torch.arange(vocab, device="cuda")
    rows = torch.stack([torch.zeros(vocab, device="cuda"), n / vocab, -n / vocab, (n % 7).float(), (n // 1000).float(), -(n % 3).float() * 0.0,
                        torch.where(n == vocab - 1, 3.0, 1.0), torch.where(n % 97 == 3, 2.0, -1.0)])
    for dtype in (F32, BF16):
        z = rows.to(dtype)
        for top in (1, 5, 32):
            _check(z, torch.arange(len(rows), device="cuda") * 31 % vocab, 1.0, top)


@pytest.mark.parametrize("vocab", [40, 1500, 40000])
def test_tokens_that_cannot_be(vocab):
    """Rows with few, one and no possible tokens, masks of the type's lowest value; certain and far-off logits."""
    for dtype in (F32, BF16):
        z = _logits(9, vocab, dtype, seed=3).t.clone()
        z[0, 5:] = -INF
        z[1] = -INF
        z[2] = -INF
        z[2, vocab - 1] = 4.0
        z[3, ::2] = torch.finfo(dtype).min
        z[4] = torch.finfo(dtype).min
        z[5, 7] = 300.0
        z[6] += 2000.0
        z[7] -= 2000.0
        ids = torch.tensor([2, 3, vocab - 1, 0, 1, 7, -1, 5, 6], device="cuda")
        r = _check(z, ids, 1.0, 8)
        assert float(r.lse[1]) == -INF and float(r.logp[1]) == -INF and float(r.entropy[1]) == 0 and int(r.top_ids[1].max()) == -1
        assert r.top_ids[2].tolist() == [vocab - 1] + [-1] * 7 and float(r.logp[2]) == 0 and float(r.entropy[2]) == 0
        assert abs(float(r.entropy[4]) - math.log(vocab)) < 1e-3
        ids[2] = 0  # a token that cannot be
        assert float(ra.ra_logprobs(z, ids).logp[2]) == -INF


@pytest.mark.parametrize("vocab", [40, 1500, 40000])
def test_non_finite_rows(vocab):
    for dtype in (F32, BF16):
        z = _logits(5, vocab, dtype, seed=4).t.clone()
        z[1, vocab // 2], z[2, 3], z[3] = NAN, INF, NAN
        z[1, 1] = -INF
        r = ra.ra_logprobs(z, torch.tensor([0, 1, 2, 3, -1], device="cuda"), entropy=True, top=3)
        for t in (r.lse, r.logp, r.entropy, r.top_logp):
            assert bool(torch.isnan(t[1:4]).all()) and bool(torch.isfinite(t[0]).all()) and bool(torch.isfinite(t[4]).all())
        assert torch.equal(r.top_ids.cpu(), alternatives64(z, 3)) and bool((r.top_ids[1:4] == -1).all())


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,vocab", [(2000, 700), (1500, 6007), (1300, 12001), (900, 20011)])
def test_several_rows_a_group(rows, vocab, dtype):
    """One, two, four and eight warps a row, each group with several rows, rows of all alignments."""
    z = _logits(rows, vocab, dtype, gap=1)
    for scale, top in ((1.0, 0), (1.1, 8), (0.9, 20), (1.0, 32)):
        _check(z.t, _ids(rows, vocab), scale, top)


@pytest.mark.parametrize("vocab", [6007, 12001])
def test_four_warps_a_row(vocab):
    test_rows_with_equal_and_ordered_logits(vocab)
    test_tokens_that_cannot_be(vocab)
    test_non_finite_rows(vocab)


def test_nothing_to_do():
    z = torch.zeros(4, 10, device="cuda")
    r = ra.ra_logprobs(z[:0], torch.zeros(0, dtype=torch.int64, device="cuda"), entropy=True, top=2)
    assert r.logp.shape == (0,) and r.top_ids.shape == (0, 2)
    r = ra.ra_logprobs(z[:, :0], torch.zeros(4, dtype=torch.int64, device="cuda"), entropy=True, top=2)
    assert not bool(r.logp.any()) and bool((r.lse == -INF).all()) and not bool(r.entropy.any()) and bool((r.top_ids == -1).all())
    r = ra.ra_logprobs(z)
    assert r.logp is None and r.entropy is None and abs(float(r.lse[0]) - math.log(10)) < 1e-6
    assert ra.ra_logprobs_grad(z[:0], None, z[:0, 0].contiguous()).shape == (0, 10)


# ---------------------------------------------------------------------------


def _check_grad(logits, ids, scale, entropy, out=None, dtype=None, seed=0, lead=0, gap=0):
    rows, vocab = logits.shape
    r = ra.ra_logprobs(logits, ids, scale=scale, entropy=True)
    gen = torch.Generator(device="cuda").manual_seed(seed + rows)
    g = torch.randn(rows, generator=gen, device="cuda")
    ge = torch.randn(rows, generator=gen, device="cuda") if entropy else None
    inside = (ids >= 0) & (ids < vocab)
    g[~inside] = NAN  # padding's counts for nothing
    s = float(torch.tensor(scale, dtype=F32))
    z, m, log_s, h, p = distribution64(logits, s)
    gd = torch.where(inside & (log_s > -INF), g.double(), 0.0).unsqueeze(1)
    want, size = -gd * p, gd.abs() * p
    hot = torch.nn.functional.one_hot(ids.long().clamp(0, vocab - 1), vocab) * gd
    want, size = want + hot, size + hot.abs()
    _, lse_bound, h_bound = _bounds(z, m, log_s, h, p)
    d = _finite((z - m.unsqueeze(1)) - _finite(log_s).unsqueeze(1))
    # p is off by its argument's error: that of lse, 8 u of |z|, |lse| and their difference, and 2^-21 for the exponential
    rel = lse_bound.unsqueeze(1) + 8 * U * (_finite(z).abs() + _finite(m + log_s).abs().unsqueeze(1) + d.abs()) + 2.0 ** -20
    bound = rel * gd.abs() * p + 4 * U * size
    if entropy:
        e = ge.double().unsqueeze(1)
        term = p * (d + h.unsqueeze(1))
        want = want - e * term
        bound = bound + e.abs() * p * ((rel + 8 * U) * (d.abs() + h.unsqueeze(1)) + rel + h_bound.unsqueeze(1))
    want, bound = want * s, bound * s
    frame = Framed(rows, vocab, dtype or logits.dtype, lead, gap) if out is None else None
    got = ra.ra_logprobs_grad(logits, ids, r.lse, g, scale=scale, entropy=r.entropy if entropy else None, grad_entropy=ge, out=frame.t if out is None else out)
    check(got, want, bound + half_step(got.dtype) * want.abs() + 2.0 ** -126, "gradient")  # the exponential flushes what is below 2^-126
    if frame is not None:
        frame.intact("gradient")
    return got


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("entropy", [False, True])
@pytest.mark.parametrize("rows,vocab", [(1, 1), (5, 2), (40, 31), (700, 257), (17, 1000), (3, 4097), (4, 32000), (3, 32001), (1, 131071)])
def test_gradient(rows, vocab, dtype, entropy):
    z = _logits(rows, vocab, dtype)
    for scale in (1.0, 0.7):
        _check_grad(z.t, _ids(rows, vocab), scale, entropy)
    _check_grad(z.t, _ids(rows, vocab, dtype=torch.int32), 1.3, entropy, dtype=F32 if dtype == BF16 else BF16)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("lead,gap,lead2,gap2", [(1, 0, 1, 0), (0, 1, 3, 2), (3, 4, 0, 0), (8, 8, 8, 8), (0, 0, 1, 1)])
def test_gradient_layouts(lead, gap, lead2, gap2, dtype):
    for rows, vocab in ((50, 300), (5, 5000)):
        z = _logits(rows, vocab, dtype, lead=lead, gap=gap)
        _check_grad(z.t, _ids(rows, vocab), 0.9, True, lead=lead2, gap=gap2)
        _check_grad(z.t, _ids(rows, vocab), 0.9, False, dtype=F32, lead=lead2, gap=gap2)
        z.intact("logits")


@pytest.mark.parametrize("vocab", [40, 1500, 40000])
def test_gradient_of_masked_rows(vocab):
    for dtype in (F32, BF16):
        z = _logits(6, vocab, dtype, seed=3).t.clone()
        z[0, 5:] = -INF
        z[1] = -INF
        z[2] = -INF
        z[2, vocab - 1] = 4.0
        z[3, ::2] = torch.finfo(dtype).min
        z[4, 7] = 300.0
        ids = torch.tensor([2, 3, vocab - 1, 0, 7, -1], device="cuda")
        for entropy in (False, True):
            got = _check_grad(z, ids, 1.0, entropy)
            assert not bool(got[1].any()) and not bool(got[0, 5:].any()) and not bool(got[2, :-1].any())
    z[0] = torch.finfo(dtype).min  # masked throughout by the type's lowest value: no gradient either
    r = ra.ra_logprobs(z, ids, entropy=True)
    e = torch.ones(6, device="cuda")
    assert not bool(ra.ra_logprobs_grad(z, ids, r.lse, e, entropy=r.entropy, grad_entropy=e)[0].any())
    z[5, 1] = NAN
    r = ra.ra_logprobs(z, ids)
    got = ra.ra_logprobs_grad(z, torch.zeros_like(ids), r.lse, torch.ones(6, device="cuda"))
    assert bool(torch.isnan(got[5]).all()) and bool(torch.isfinite(got[:5]).all())


def test_gradient_in_place_and_without_parts():
    for vocab in (1000, 1001):
        z = _logits(30, vocab, BF16).t.clone()
        ids = _ids(30, vocab)
        want = _check_grad(z, ids, 1.0, False)
        assert torch.equal(_check_grad(z, ids, 1.0, False, out=z.clone()), want)
        r = ra.ra_logprobs(z, ids, entropy=True)
        g = torch.where((ids >= 0) & (ids < vocab), 0.5, NAN)
        held = z.clone()
        assert ra.ra_logprobs_grad(held, ids, r.lse, g, out=held) is held and torch.equal(held, ra.ra_logprobs_grad(z, ids, r.lse, g))
        e = torch.full((30,), 2.0, device="cuda")
        both = ra.ra_logprobs_grad(z, ids, r.lse, torch.zeros(30, device="cuda"), entropy=r.entropy, grad_entropy=e)
        assert torch.equal(ra.ra_logprobs_grad(z, None, r.lse, entropy=r.entropy, grad_entropy=e), both)
        assert not bool(ra.ra_logprobs_grad(z, None, r.lse).any())


def test_gradient_against_differences():
    rows, vocab, h, scale = 3, 12, 1e-4, 0.8
    z = _logits(rows, vocab, F32, s=1.0).t.clone()
    z[1, 4] = -INF
    ids = torch.tensor([3, 0, -1], device="cuda")
    g, ge = torch.tensor([1.5, -0.5, 9.0], device="cuda"), torch.tensor([0.3, 0.7, -0.4], device="cuda")
    r = ra.ra_logprobs(z, ids, scale=scale, entropy=True)
    got = ra.ra_logprobs_grad(z, ids, r.lse, g, scale=scale, entropy=r.entropy, grad_entropy=ge).double()

    def loss(v):
        y = v * scale
        lse = torch.logsumexp(y, 1)
        p = torch.exp(y - lse.unsqueeze(1))
        ent = lse - torch.where(p > 0, p * y, 0.0).sum(1)
        lp = torch.where(ids >= 0, y.gather(1, ids.clamp(min=0).unsqueeze(1)).squeeze(1) - lse, 0.0)
        return (g.double() * lp + ge.double() * ent).sum()

    for a in range(rows):
        for b in range(vocab):
            up, down = z.double(), z.double()
            up[a, b] += h
            down[a, b] -= h
            if torch.isfinite(z[a, b]):
                assert abs(float((loss(up) - loss(down)) / (2 * h)) - float(got[a, b])) < 2e-6  # h^2 and 40 u of values near 1


def test_streams_and_graphs():
    z, ids = _logits(64, 5000, BF16).t, _ids(64, 5000)
    want = ra.ra_logprobs(z, ids, entropy=True, top=4)
    torch.cuda.synchronize()
    got = [ra.ra_logprobs(z, ids, entropy=True, top=4, stream=s) for s in (torch.cuda.Stream(), torch.cuda.Stream())]
    torch.cuda.synchronize()
    for r in got:
        for name in ra.LogProbs.__slots__:
            assert torch.equal(getattr(r, name), getattr(want, name))
    g = torch.ones(64, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = ra.ra_logprobs(z, ids, entropy=True, top=4)
        d = ra.ra_logprobs_grad(z, ids, r.lse, g)
    z.mul_(0.5)
    graph.replay()
    graph.replay()
    want = ra.ra_logprobs(z, ids, entropy=True, top=4)
    assert torch.equal(r.top_ids, want.top_ids) and torch.equal(r.lse, want.lse) and torch.equal(d, ra.ra_logprobs_grad(z, ids, want.lse, g))


def test_past_32_bit_offsets():
    rows, vocab = 70_001, 32000  # 2.24 G values
    z = torch.zeros(rows, vocab, dtype=BF16, device="cuda")
    ids = torch.full((rows,), vocab - 1, device="cuda")
    z[-1] = _logits(1, vocab, BF16).t[0]
    r = ra.ra_logprobs(z, ids, top=2)
    z1, m, log_s, _, p = distribution64(z[-1:], 1.0)
    assert torch.equal(r.top_ids[-1:].cpu(), alternatives64(z[-1:], 2)) and abs(float(r.lse[-1]) - float(m + log_s)) < 1e-5
    assert abs(float(r.logp[-1]) - float(z1[0, -1] - m - log_s)) < 1e-5 and abs(float(r.lse[-2]) - math.log(vocab)) < 1e-5
    g = torch.ones(rows, device="cuda")
    last = ra.ra_logprobs_grad(z[-1:], ids[-1:], r.lse[-1:], g[-1:])
    ra.ra_logprobs_grad(z, ids, r.lse, g, out=z)
    assert torch.equal(z[-1:], last)
    del z
    torch.cuda.empty_cache()


def test_refusals():
    z, i = torch.zeros(4, 8, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")
    v = torch.zeros(4, device="cuda")
    for call in (lambda: ra.ra_logprobs(z[0], i), lambda: ra.ra_logprobs(z, i[:3]), lambda: ra.ra_logprobs(z, i.cpu()), lambda: ra.ra_logprobs(z, i, top=33),
                 lambda: ra.ra_logprobs(z, i, top=-1), lambda: ra.ra_logprobs(z.t(), i), lambda: ra.ra_logprobs_grad(z, i, v[:3], v),
                 lambda: ra.ra_logprobs_grad(z, i, v, v[:3]), lambda: ra.ra_logprobs_grad(z, i, v, v, grad_entropy=v),
                 lambda: ra.ra_logprobs_grad(z, i[:2], v, v), lambda: ra.ra_logprobs_grad(z, i, v, v, out=z[:2])):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: ra.ra_logprobs(z.half(), i), lambda: ra.ra_logprobs(z, i.float()), lambda: ra.ra_logprobs_grad(z, i, v.double(), v),
                 lambda: ra.ra_logprobs_grad(z, i, v, v.bfloat16()), lambda: ra.ra_logprobs_grad(z, i, v, v, dtype=torch.float16)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(ra.RaError, match="OVERLAP"):
        ra.ra_logprobs_grad(z[:2], i[:2], v[:2], v[:2], out=z[1:3])
    with pytest.raises(ra.RaError, match="INVALID"):
        ra.ra_logprobs(z, i, scale=0.0)
