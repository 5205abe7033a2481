"""ra_embedding_lookup and ra_embedding_grad against plain forms in 64 bits."""
from __future__ import annotations

import pytest
import torch

import gradient_ring_all_gb300 as ra
from operator_reference import U, Framed, check, rounding

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from gradient_ring_all_gb300 import build
    build.build()
    ra.load()


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _ids(kind, count, vocab, seed, dtype=torch.int64):
    g = _gen(seed)
    if kind == "one":
        ids = torch.full((count,), vocab // 2, device="cuda")
    elif kind == "falling":
        ids = (vocab - 1 - torch.arange(count, device="cuda")) % vocab
    elif kind == "none":
        ids = torch.where(torch.arange(count, device="cuda") % 2 == 0, -1, vocab)
    elif kind == "few":  # three ids, one of them the last, and padding
        ids = torch.tensor([0, vocab - 1, vocab // 3, -100], device="cuda")[torch.randint(0, 4, (count,), generator=g, device="cuda")]
    else:
        ids = torch.randint(-1, vocab + 1, (count,), generator=g, device="cuda")
    return ids.to(dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("id_type", [torch.int32, torch.int64])
@pytest.mark.parametrize("tokens,vocab,d,lead,gap", [
    (1, 1, 1, 0, 0), (1, 7, 2048, 0, 0), (37, 1000, 509, 0, 0), (64, 50, 512, 8, 8), (300, 3, 130, 1, 1), (5, 9, 4096, 0, 2),
    (2049, 257, 24, 4, 4)])
def test_lookup(tokens, vocab, d, lead, gap, dtype, id_type):
    table = Framed(vocab, d, dtype, lead, gap).fill(torch.randn(vocab, d, generator=_gen(1), device="cuda"))
    ids = _ids("random", tokens, vocab, 2, id_type)
    out = Framed(tokens, d, dtype, lead, gap)
    scale = 3.3
    ra.ra_embedding_lookup(table.t, ids, scale=scale, out=out.t)
    inside = (ids >= 0) & (ids < vocab)
    want = (table.t.float()[ids.clamp(0, vocab - 1).long()] * torch.tensor(scale, device="cuda")).to(dtype)
    want[~inside] = 0
    assert torch.equal(out.t, want)
    out.intact("lookup")


def test_lookup_of_nothing_and_non_finite_rows():
    table = torch.randn(4, 8, device="cuda")
    table[2] = float("nan")
    table[3, 0] = float("inf")
    assert ra.ra_embedding_lookup(table, torch.empty(0, dtype=torch.int64, device="cuda")).shape == (0, 8)
    out = ra.ra_embedding_lookup(table, torch.tensor([2, 3, -1, 4], device="cuda"))
    assert bool(torch.isnan(out[0]).all()) and float(out[1, 0]) == float("inf") and not bool(out[2:].any())


def test_lookup_past_32_bit_offsets():
    # 2^21 + 3 rows of 1040 bf16 values: the last row starts beyond 2^31 elements
    vocab, d = (1 << 21) + 3, 1040
    table = torch.empty(vocab, d, dtype=BF16, device="cuda")
    rows = torch.tensor([0, 1, vocab // 2, vocab - 2, vocab - 1], device="cuda")
    table[rows] = torch.randn(5, d, generator=_gen(3), device="cuda").to(BF16)
    assert torch.equal(ra.ra_embedding_lookup(table, rows), table[rows])
    g = torch.randn(5, d, generator=_gen(4), device="cuda").to(BF16)
    table.fill_(1)
    ra.ra_embedding_grad(g, rows, vocab, out=table, accumulate=True)
    assert torch.equal(table[rows], (1 + g.float()).to(BF16))
    ra.ra_embedding_grad(g, rows, vocab, out=table)
    assert torch.equal(table[rows], g) and not bool(table[2:vocab // 2].any()) and not bool(table[vocab // 2 + 1:vocab - 2].any())
    del table
    torch.cuda.empty_cache()


def _grad64(grad, ids, vocab, scale):
    """(the sum in 64 bits, the sum of magnitudes, tokens per id)"""
    keep = (ids >= 0) & (ids < vocab)
    ids, g = ids[keep].long(), grad[keep].double()
    s = torch.zeros(vocab, grad.shape[1], dtype=torch.float64, device="cuda")
    a = torch.zeros_like(s)
    n = torch.zeros(vocab, 1, dtype=torch.float64, device="cuda")
    s.index_add_(0, ids, g)
    a.index_add_(0, ids, g.abs())
    n.index_add_(0, ids, torch.ones(ids.shape[0], 1, dtype=torch.float64, device="cuda"))
    return s * scale, a * abs(scale), n


TOKENS = [1, 2, 31, 32, 33, 64, 65, 97, 1000, 4096, 4097, 9000]


@pytest.mark.parametrize("kind", ["random", "one", "falling", "none", "few"])
@pytest.mark.parametrize("tokens", TOKENS)
def test_grad_by_ids(kind, tokens):
    for vocab, d in ((1, 8), (255, 24), (256, 33), (5000, 40)):
        ids = _ids(kind, tokens, vocab, tokens)
        grad = torch.randn(tokens, d, generator=_gen(tokens), device="cuda")
        grad[(ids < 0) | (ids >= vocab)] = float("nan")  # padding's rows count for nothing
        got = ra.ra_embedding_grad(grad, ids, vocab, scale=0.7)
        want, size, n = _grad64(grad, ids, vocab, float(torch.tensor(0.7)))
        check(got, want, 2 * (n + 2) * U * size, "%s vocab %d" % (kind, vocab))
        assert not bool(got[(n == 0).squeeze(1)].any())
        assert torch.equal(got, ra.ra_embedding_grad(grad, ids, vocab, scale=0.7))  # the same bits again


@pytest.mark.parametrize("in_type", [F32, BF16])
@pytest.mark.parametrize("out_type", [F32, BF16])
@pytest.mark.parametrize("id_type", [torch.int32, torch.int64])
@pytest.mark.parametrize("d,lead,gap", [(1, 0, 0), (7, 0, 0), (64, 8, 8), (1022, 0, 0), (2048, 0, 0), (100, 2, 2), (130, 1, 0)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_grad_by_layout(in_type, out_type, id_type, d, lead, gap, accumulate):
    tokens, vocab, scale = 700, 300, -2.5
    ids = _ids("few" if d % 2 else "random", tokens, vocab, d, id_type)
    grad = Framed(tokens, d, in_type, lead, gap).fill(torch.randn(tokens, d, generator=_gen(d), device="cuda"))
    old = torch.randn(vocab, d, generator=_gen(d + 1), device="cuda").to(out_type)
    out = Framed(vocab, d, out_type, lead, gap).fill(old if accumulate else torch.full_like(old, float("nan")))
    ra.ra_embedding_grad(grad.t, ids, vocab, scale=scale, out=out.t, accumulate=accumulate)
    want, size, n = _grad64(grad.t, ids, vocab, scale)
    if accumulate:
        want = want + old.double()
        size = size + old.double().abs()
        untouched = (n == 0).squeeze(1)
        assert torch.equal(out.t[untouched], old[untouched])
    check(out.t, want, 2 * (n + 3) * U * size + rounding(out_type) * want.abs())
    out.intact("grad")


def test_grad_with_a_wide_vocabulary():
    # ids that need three sorting passes, and pieces of one id over many blocks
    vocab, tokens, d = 70_000, 20_000, 16
    ids = _ids("random", tokens, vocab, 8)
    ids[5000:12_000] = 69_999
    grad = torch.randn(tokens, d, generator=_gen(9), device="cuda")
    want, size, n = _grad64(grad, ids, vocab, 1.0)
    check(ra.ra_embedding_grad(grad, ids, vocab), want, 2 * (n + 2) * U * size)


@pytest.mark.parametrize("tokens", [16_384, 16_385, 131_072, 131_073, 300_001])
def test_grad_by_number_of_tokens(tokens):
    """One block's sort and the tiled one: the sums are exact here (small whole numbers)."""
    for vocab in (200, 40_000):
        ids = _ids("random", tokens, vocab, tokens)
        ids[tokens // 3: tokens // 2] = 7
        grad = torch.randint(-3, 4, (tokens, 5), generator=_gen(tokens), device="cuda").float()
        want, _, _ = _grad64(grad, ids, vocab, 1.0)
        assert torch.equal(ra.ra_embedding_grad(grad, ids, vocab).double(), want)


def test_grad_of_no_tokens():
    ids = torch.empty(0, dtype=torch.int64, device="cuda")
    g = torch.empty(0, 8, device="cuda")
    out = torch.full((5, 8), 3.0, device="cuda")
    ra.ra_embedding_grad(g, ids, 5, out=out, accumulate=True)
    assert bool((out == 3).all())
    ra.ra_embedding_grad(g, ids, 5, out=out)
    assert not bool(out.any())
    assert ra.ra_embedding_grad(g, ids, 0).shape == (0, 8)


def test_grad_against_differences():
    # L = sum(c * lookup(E)); dL/dE by central differences in 64 bits
    vocab, d, tokens, scale, h = 6, 3, 11, 1.5, 1e-4
    ids = _ids("random", tokens, vocab, 12)
    c = torch.randn(tokens, d, generator=_gen(13), device="cuda")
    table = torch.randn(vocab, d, generator=_gen(14), device="cuda", dtype=torch.float64)

    def loss(e):
        rows = e[ids.clamp(0, vocab - 1)] * scale
        rows[(ids < 0) | (ids >= vocab)] = 0
        return (c.double() * rows).sum()

    got = ra.ra_embedding_grad(c, ids, vocab, scale=scale).double()
    for v in range(vocab):
        for j in range(d):
            up, down = table.clone(), table.clone()
            up[v, j] += h
            down[v, j] -= h
            diff = float((loss(up) - loss(down)) / (2 * h))
            # the loss is linear in E: what is left is the differences' own rounding and the kernel's
            assert abs(float(got[v, j]) - diff) <= 1e-9 / h * 1e-2 + 2 * (tokens + 2) * U * float(c.abs().sum()) * scale


def test_refusals():
    t = torch.zeros(8, 16, device="cuda")
    i = torch.zeros(4, dtype=torch.int64, device="cuda")
    with pytest.raises(TypeError):
        ra.ra_embedding_lookup(t, i.float())
    with pytest.raises(ValueError):
        ra.ra_embedding_lookup(t, i.cpu())
    with pytest.raises(ValueError):
        ra.ra_embedding_lookup(t, torch.zeros(8, dtype=torch.int64, device="cuda")[::2])
    with pytest.raises(TypeError):
        ra.ra_embedding_lookup(t, i, out=torch.zeros(4, 16, dtype=BF16, device="cuda"))
    with pytest.raises(ra.RaError, match="OVERLAP"):
        ra.ra_embedding_lookup(t, i, out=t[:4])
    with pytest.raises(ValueError):
        ra.ra_embedding_grad(t, i, 8)
    with pytest.raises(ValueError):
        ra.ra_embedding_grad(t[:4], i, 8, accumulate=True)
    with pytest.raises(ValueError):
        ra.ra_embedding_grad(t[:4], i, 8, out=torch.zeros(9, 16, device="cuda"))
    with pytest.raises(ra.RaError, match="OVERLAP"):
        ra.ra_embedding_grad(t[:4], i, 8, out=t)
    with pytest.raises(ra.RaError, match="INVALID"):
        ra.ra_embedding_grad(t[:4], i, 8, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
