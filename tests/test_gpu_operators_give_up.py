"""The products' waits are bounded: with a block that makes no copies every wait
on them runs out, the call reports it, returns, and leaves what that block would
have stored as it was.  No fault, no hang: the copies are simply not made."""
from __future__ import annotations

import pytest
import torch

import gradient_ring_all_gb300 as ra
from operator_reference import check, rounding, sum_bound

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
LIMIT_US = 20_000
HELD = -1e30  # what outputs hold before the call; far outside every result


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from gradient_ring_all_gb300 import build
    build.build()
    ra.load()


def _normal(seed, *shape, dtype=BF16, s=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * s).to(dtype)


def _timed_out():
    torch.cuda.synchronize()
    return ra.ra_check_device_errors() == ra.RA_ERR_TIMEOUT


def _held_or_right(got, want, bound, most):
    """Each value is the former one or the product's; between one and `most` of them are the former ones."""
    held = got == torch.full((), HELD, dtype=got.dtype, device="cuda")
    check(got[~held], want[~held], bound[~held])
    assert 0 < int(held.sum()) <= most, (int(held.sum()), most)


# (m, k, n): single blocks of 64 and 128 columns; pairs of 128 and 256; no block or pair has more than two tiles
WHOLE = [(300, 200, 130), (2000, 130, 1500), (1000, 640, 2000), (4096, 512, 1100)]


@pytest.mark.parametrize("out_type", [BF16, F32])
@pytest.mark.parametrize("m,k,n", WHOLE)
@pytest.mark.parametrize("block", [0, 1, 4])
def test_a_block_that_gives_up(block, m, k, n, out_type):
    x, w = _normal(1, m, k), _normal(2, k, n, s=k ** -0.5)
    want, size = x.double() @ w.double(), x.double().abs() @ w.double().abs()
    bound = sum_bound(k) * size + rounding(out_type) * want.abs()
    out = torch.full((m, n), HELD, dtype=out_type, device="cuda")
    assert ra.ra_check_device_errors() == ra.RA_OK
    ra.ra_selftest_linear_stall(block, LIMIT_US)
    ra.ra_linear(x, w, out=out)
    assert _timed_out()
    _held_or_right(out, want, bound, 2 * 256 * 256)
    # the next call is an ordinary one
    check(ra.ra_linear(x, w, dtype=out_type), want, bound)
    assert ra.ra_check_device_errors() == ra.RA_OK
    for product in (lambda o: ra.ra_linear_dgrad(x, wt, out=o), lambda o: ra.ra_linear_wgrad(xt, w, out=o)):
        xt, wt = x.t().contiguous(), w.t().contiguous()
        out.fill_(HELD)
        ra.ra_selftest_linear_stall(block, LIMIT_US)
        product(out)
        assert _timed_out()
        _held_or_right(out, want, bound, 2 * 256 * 256)
        product(out)
        check(out, want, bound)


def test_limits_out_of_range():
    for block, limit in ((-1, 10), (0, 0), (0, -5), (0, 10_000_001)):
        with pytest.raises(ra.RaError):
            ra.ra_selftest_linear_stall(block, limit)


@pytest.mark.parametrize("out_type", [BF16, F32])
@pytest.mark.parametrize("m,k,n", [(256, 300, 130), (512, 2000, 2000), (256, 8192, 4000), (100, 4100, 8192)])
@pytest.mark.parametrize("block", [0, 1, 76])
def test_a_block_that_gives_up_beside_column_sums(block, m, k, n, out_type):
    """The bias gradient's sums wait for no copies: they are whole, also where a block has several of the first row's tiles and
    gives up at the first (the epilogue warps' common barriers must all be behind them by then)."""
    x, dy = _normal(1, m, k), _normal(2, m, n)
    out, db = torch.full((k, n), HELD, dtype=out_type, device="cuda"), torch.full((n,), HELD, device="cuda")
    ra.ra_selftest_linear_stall(block, LIMIT_US)
    ra.ra_linear_wgrad(x, dy, out=out, bias_grad=db)
    timed_out = _timed_out()
    want, size = x.double().t() @ dy.double(), x.double().t().abs() @ dy.double().abs()
    bound = sum_bound(m) * size + rounding(out_type) * want.abs()
    check(db, dy.double().sum(0), sum_bound(m) * dy.double().abs().sum(0))
    if timed_out:
        _held_or_right(out, want, bound, 8 * 256 * 256)
    else:  # the grid has no such block
        check(out, want, bound)
    assert timed_out or block == 76


# (m, k, n): clusters that split k, of single blocks (with few rows, and with a tile's), and of two and four pairs
SPLIT = [(16, 2048, 2048), (3, 4096, 200), (1, 1100, 4000), (120, 4096, 4096), (256, 1024, 1024), (257, 3210, 2081), (300, 4104, 328)]


@pytest.mark.parametrize("out_type", [BF16, F32])
@pytest.mark.parametrize("m,k,n", SPLIT)
@pytest.mark.parametrize("block", [0, 1, 2, 3, 7])
def test_a_block_of_a_cluster_that_gives_up(block, m, k, n, out_type):
    """No block of the cluster stores a sum in which that block's share is missing."""
    w, bias = _normal(2, k, n, s=k ** -0.5), _normal(3, n, dtype=F32)
    for rows in sorted({m, max(m, 2)}):  # a single row has a kernel without copies
        x = _normal(1, rows, k)
        z, size = x.double() @ w.double(), x.double().abs() @ w.double().abs()
        want, bound = z + bias.double(), sum_bound(k + 1) * (size + bias.double().abs())
        bound = bound + rounding(out_type) * want.abs()
        out = torch.full((rows, n), HELD, dtype=out_type, device="cuda")
        kept = ra.Checkpoint8(rows, n)
        kept.q.fill_(77)
        kept.e.fill_(3)
        ra.ra_selftest_linear_stall(block, LIMIT_US)
        if rows > 1:
            ra.ra_linear(x, w, bias=bias, save=kept, out=out)
            assert _timed_out()
            _held_or_right(out, want, bound, 256 * 128)
            held = (out == torch.full((), HELD, dtype=out_type, device="cuda")).any(0).int()
            held = torch.nn.functional.pad(held, (0, -n % 32)).view(-1, 32).any(1)
            tops = kept.e == 3  # no group of these sums has such a step
            assert torch.equal(tops.any(0), held)
            assert bool((kept.q.view(rows, -1, 32)[tops] == 77).all())
        for product in (lambda o: ra.ra_linear_dgrad(x, wt, out=o), lambda o: ra.ra_linear_wgrad(xt, w, out=o)):
            xt, wt = x.t().contiguous(), w.t().contiguous()
            out.fill_(HELD)
            ra.ra_selftest_linear_stall(block, LIMIT_US)
            product(out)
            timed_out = _timed_out()
            if timed_out:
                _held_or_right(out, z, sum_bound(k) * size + rounding(out_type) * z.abs(), 256 * 128)
            product(out)
            check(out, z, sum_bound(k) * size + rounding(out_type) * z.abs())


@pytest.mark.parametrize("out_type", [BF16, F32])
@pytest.mark.parametrize("block", [0, 1, 30, 60, 151])
def test_a_part_of_a_tile_that_is_not_made(block, out_type):
    """Tiles whose sums are made in parts along k and joined afterwards: without one of the parts none of the tile is stored."""
    from gradient_ring_all_gb300 import operators
    m, k, n = 2500, 4100, 2200
    x, w = _normal(1, m, 4104)[:, :k], _normal(2, k, n, s=k ** -0.5)
    lib = operators._load()
    need = lib.ra_linear_split_bytes(m, n, k)
    assert need > 0
    want, size = x.double() @ w.double(), x.double().abs() @ w.double().abs()
    bound = sum_bound(k) * size + rounding(out_type) * want.abs()
    out = torch.full((m, n), HELD, dtype=out_type, device="cuda")
    workspace = torch.empty(need, dtype=torch.uint8, device="cuda")
    for product in (lambda: ra.ra_linear(x, w, out=out, workspace=workspace), lambda: ra.ra_linear_dgrad(x, wt, out=out, workspace=workspace),
                    lambda: ra.ra_linear_wgrad(xt, w, out=out, workspace=workspace)):
        xt, wt = torch.empty(k, 2504, dtype=BF16, device="cuda")[:, :m].copy_(x.t()), torch.empty(n, 4104, dtype=BF16, device="cuda")[:, :k].copy_(w.t())
        product()  # right sums of every part lie in the workspace
        check(out, want, bound)
        out.fill_(HELD)
        ra.ra_selftest_linear_stall(block, LIMIT_US)
        product()
        assert _timed_out()
        # the pair's first tile, and the tile of its part
        _held_or_right(out, want, bound, 2 * 256 * 256)
        product()
        check(out, want, bound)
