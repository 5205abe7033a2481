"""ra_dropout against the mask made on the host and the same two roundings."""
from __future__ import annotations

import pytest
import torch

import gradient_ring_all_gb300 as ra
from block_reference import keep_mask
from operator_reference import Framed

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
SEED = 0xFEDCBA9876543210


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from gradient_ring_all_gb300 import build
    build.build()
    ra.load()


def _normal(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


def _want(x, p, seed, site=0, first_row=0, residual=None, dtype=None):
    """Each operation in binary32, as the kernel rounds: the scaled value, then the sum, then the type."""
    keep = keep_mask(*x.shape, p, seed, site, first_row).cuda()
    t = round(65536 * p)
    scale = torch.tensor(65536 / (65536 - t) if t < 65536 else 0.0, device="cuda")
    y = torch.where(keep, x.float() * scale, torch.zeros((), device="cuda"))
    if residual is not None:
        y = y + residual.float()
    return y.to(dtype or x.dtype)


@pytest.mark.parametrize("x_type,y_type,res_type", [(F32, F32, None), (BF16, BF16, None), (BF16, F32, F32), (F32, BF16, BF16), (F32, F32, F32), (BF16, BF16, BF16)])
@pytest.mark.parametrize("rows,cols,lead,gap", [(1, 1, 0, 0), (1, 8, 0, 0), (3, 7, 0, 0), (5, 2048, 0, 0), (64, 264, 8, 8), (33, 257, 1, 2), (130, 40, 0, 4),
                                                (7, 4104, 0, 0), (1, 70001, 3, 0), (2000, 16, 0, 0)])
def test_values_and_mask(rows, cols, lead, gap, x_type, y_type, res_type):
    x = Framed(rows, cols, x_type, lead, gap).fill(_normal(1, rows, cols))
    res = None if res_type is None else Framed(rows, cols, res_type, lead, gap).fill(_normal(2, rows, cols))
    out = Framed(rows, cols, y_type, lead, gap)
    ra.ra_dropout(x.t, 0.3, SEED, site=7, first_row=11, residual=None if res is None else res.t, out=out.t)
    assert torch.equal(out.t, _want(x.t, 0.3, SEED, 7, 11, None if res is None else res.t, y_type))
    out.intact("dropout")
    x.intact("x")


@pytest.mark.parametrize("p", [0.0, 1e-6, 0.25, 0.5, 0.999, 1 - 2.0 ** -17, 1.0])
def test_probabilities(p):
    x = _normal(3, 50, 72)
    x[0, 0], x[1, 1] = float("nan"), float("inf")
    got, want = ra.ra_dropout(x, p, 1), _want(x, p, 1)
    assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(), want.nan_to_num())
    if p == 0.0:
        assert torch.equal(got[2:], x[2:])
    if p == 1.0:
        assert not bool(got.any())  # dropped values count as 0, whatever they hold


def test_micro_batches_and_slices_take_their_part_of_the_mask():
    x = _normal(4, 100, 88).to(BF16)
    whole = ra.ra_dropout(x, 0.4, SEED, site=3)
    for a, b in ((0, 1), (1, 50), (50, 100)):
        assert torch.equal(ra.ra_dropout(x[a:b], 0.4, SEED, site=3, first_row=a), whole[a:b])
    assert torch.equal(ra.ra_dropout(x[:, :35], 0.4, SEED, site=3), whole[:, :35])
    # rows beyond 2^32 and 2^62
    for first in ((1 << 32) - 2, (1 << 62) + 5):
        assert torch.equal(ra.ra_dropout(x[:5], 0.4, SEED, first_row=first), _want(x[:5], 0.4, SEED, 0, first))
    assert not torch.equal(ra.ra_dropout(x, 0.4, SEED, site=4), whole) and not torch.equal(ra.ra_dropout(x, 0.4, SEED ^ (1 << 63), site=3), whole)


@pytest.mark.parametrize("cols", [64, 63])
def test_the_gradient_is_the_same_call(cols):
    """d/dx of sum(c * dropout(x)) is dropout(c): what reaches a dropped value is 0; checked against differences in 64 bits."""
    x, c = _normal(5, 20, cols), _normal(6, 20, cols)
    g = ra.ra_dropout(c, 0.5, 9)
    keep = keep_mask(20, cols, 0.5, 9).cuda()
    loss = lambda v: (c.double() * torch.where(keep, v * 2.0, 0.0)).sum()  # noqa: E731
    for r, k in ((0, 0), (3, 5), (19, cols - 1), (7, 30)):
        up, down = x.double(), x.double()
        up[r, k] += 1e-3
        down[r, k] -= 1e-3
        assert abs(float((loss(up) - loss(down)) / 2e-3) - float(g[r, k])) < 1e-9  # linear: what is left is 64-bit rounding over the step


def test_in_place_and_shared_arrays():
    for cols in (64, 65):
        x, r = _normal(7, 30, cols), _normal(8, 30, cols)
        want = ra.ra_dropout(x, 0.2, 5, residual=r)
        a, b = x.clone(), r.clone()
        assert ra.ra_dropout(a, 0.2, 5, residual=r, out=a) is a and torch.equal(a, want)
        assert torch.equal(ra.ra_dropout(x, 0.2, 5, residual=b, out=b), want)
        c = x.clone()
        assert torch.equal(ra.ra_dropout(c, 0.2, 5, residual=c, out=c), ra.ra_dropout(x, 0.2, 5, residual=x))
        both = torch.zeros(30, 2 * cols, device="cuda")
        both[:, :cols] = x
        ra.ra_dropout(both[:, :cols], 0.2, 5, residual=r, out=both[:, cols:])
        assert torch.equal(both[:, cols:], want) and torch.equal(both[:, :cols], x)


def test_a_seed_in_device_memory_and_a_captured_call():
    x = _normal(9, 40, 128)
    seed = torch.tensor([77], dtype=torch.int64, device="cuda")
    assert torch.equal(ra.ra_dropout(x, 0.5, seed), ra.ra_dropout(x, 0.5, 77))
    seed.fill_(-1)
    assert torch.equal(ra.ra_dropout(x, 0.5, seed), ra.ra_dropout(x, 0.5, 2 ** 64 - 1))
    out = torch.empty_like(x)
    g = torch.cuda.CUDAGraph()
    seed.fill_(5)
    with torch.cuda.graph(g):
        ra.ra_dropout(x, 0.5, seed, out=out)
        seed.add_(1)
    for k in range(3):  # each replay takes the next mask
        g.replay()
        assert torch.equal(out, ra.ra_dropout(x, 0.5, 5 + k))
    # two calls at once, on streams of their own
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    ya, yb = ra.ra_dropout(x, 0.5, 1, stream=a), ra.ra_dropout(x, 0.5, 2, stream=b)
    torch.cuda.synchronize()
    assert torch.equal(ya, ra.ra_dropout(x, 0.5, 1)) and torch.equal(yb, ra.ra_dropout(x, 0.5, 2))


def test_past_32_bit_offsets():
    rows, cols = (1 << 21) + 3, 1040  # 2.18 G values
    x = torch.ones(rows, cols, dtype=BF16, device="cuda")
    ra.ra_dropout(x, 0.5, 3, out=x)
    for a in (0, rows // 2, rows - 2):
        assert torch.equal(x[a:a + 2], _want(torch.ones(2, cols, device="cuda"), 0.5, 3, 0, a).to(BF16))
    y = x.view(-1)[1:1 + (rows - 1) * cols].view(rows - 1, cols)  # the kernel of any alignment
    y.fill_(1)
    ra.ra_dropout(y, 0.5, 4, out=y)
    assert torch.equal(y[-2:], _want(torch.ones(2, cols, device="cuda"), 0.5, 4, 0, rows - 3).to(BF16))
    del x, y
    torch.cuda.empty_cache()


def test_empty_and_refused():
    x = torch.zeros(4, 8, device="cuda")
    assert ra.ra_dropout(x[:0], 0.5, 1).shape == (0, 8) and ra.ra_dropout(x[:, :0], 0.5, 1).shape == (4, 0)
    for kw in (dict(p=-0.1), dict(p=1.1), dict(seed=-1), dict(seed=1 << 64), dict(site=-1), dict(site=1 << 32), dict(first_row=-1), dict(residual=x[:2]),
               dict(out=x[:, :4]), dict(residual=x.cpu()), dict(seed=torch.zeros(1, dtype=torch.int64))):
        with pytest.raises(ValueError):
            ra.ra_dropout(x, **{"p": 0.5, "seed": 1, **kw})
    for kw in (dict(seed=torch.zeros(2, dtype=torch.int64, device="cuda")), dict(seed=torch.zeros(1, device="cuda")), dict(residual=x.double()),
               dict(dtype=torch.float16)):
        with pytest.raises(TypeError):
            ra.ra_dropout(x, **{"p": 0.5, "seed": 1, **kw})
    with pytest.raises(ra.RaError, match="OVERLAP"):
        ra.ra_dropout(x[:2], 0.5, 1, out=x[1:3])
