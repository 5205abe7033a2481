"""ra_checkpoint8_pack / ra_checkpoint8_unpack against their definition in 64
bits: the stored bytes are equal, the restored values exact."""
from __future__ import annotations

import pytest
import torch

import gradient_ring_all_gb300 as ra
from operator_reference import Framed, act64, check, pack64, power64, rounding, values64

pytestmark = pytest.mark.gpu

SHAPES = [(1, 1), (1, 31), (1, 32), (2, 33), (3, 64), (7, 96), (5, 1001), (64, 256), (129, 520), (1, 40_000), (4096, 16)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from gradient_ring_all_gb300 import build
    build.build()
    ra.load()


def _x(rows, cols, dtype, seed, lead=0, gap=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    v = torch.randn(rows, cols, generator=g, device="cuda") * torch.exp2(torch.randint(-20, 20, (rows, 1), generator=g, device="cuda").float())
    return Framed(rows, cols, dtype, lead, gap).fill(v.to(dtype))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("lead,gap", [(0, 0), (8, 8), (1, 2), (0, 3)])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_bytes_and_values(rows, cols, lead, gap, dtype):
    x = _x(rows, cols, dtype, rows * 1000 + cols, lead, gap)
    kept = ra.ra_checkpoint8_pack(x.t)
    q, e = pack64(x.t)
    assert torch.equal(kept.e, e) and torch.equal(kept.q, q)
    want = values64(q, e, cols)
    half = power64(e.to(torch.int64) - 128).repeat_interleave(32, 1)[:, :cols]
    assert bool(((want - x.t.double()).abs() <= half).all())  # the nearest whole number of steps
    for out_type in (torch.bfloat16, torch.float32):
        out = Framed(rows, cols, out_type, lead, gap)
        ra.ra_checkpoint8_unpack(kept, out=out.t)
        assert torch.equal(out.t.double(), want)  # exact in either type
        out.intact("unpack")
    x.intact("pack")


@pytest.mark.parametrize("act", ["relu", "gelu", "silu"])
@pytest.mark.parametrize("cols", [1, 37, 64])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_restored_through_an_activation(act, cols, dtype):
    x = torch.linspace(-12, 12, 50 * cols, device="cuda").view(50, cols)
    kept = ra.ra_checkpoint8_pack(x)
    z = values64(kept.q, kept.e, cols)
    want = act64(z, act)
    got = ra.ra_checkpoint8_unpack(kept, act=act, dtype=dtype)
    check(got, want, 2.0 ** -20 * z.abs() + rounding(dtype) * want.abs(), act)


def _group(values, dtype=torch.float32):
    v = torch.zeros(1, 32, dtype=dtype, device="cuda")
    v[0, :len(values)] = torch.tensor(values, dtype=dtype, device="cuda")
    return v


@pytest.mark.parametrize("values", [
    [0.0], [-0.0, 0.0], [1.0], [-1.0, 0.5], [1.9921875], [1.9921874], [1.0, 1 / 128, 3 / 128, 5 / 128],
    [3.4028234663852886e38, -3.4028234663852886e38], [1e-45], [-1e-45, 1e-40], [1.1754943508222875e-38], [2.0 ** -119], [2.0 ** -121],
    [127.5, 0.5, 1.5, 2.5], [127.49, 0.49]])
def test_edges_of_a_group(values):
    x = _group(values)
    kept = ra.ra_checkpoint8_pack(x)
    q, e = pack64(x)
    assert torch.equal(kept.e, e) and torch.equal(kept.q, q)
    assert int(kept.q.abs().max()) <= 127
    assert torch.equal(ra.ra_checkpoint8_unpack(kept, dtype=torch.float32).double(), values64(q, e, 32))


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("cols,lead", [(96, 0), (70, 0), (70, 1)])
def test_a_group_with_a_non_finite_value_reads_back_as_nan(bad, dtype, cols, lead):
    x = _x(3, cols, dtype, 5, lead).t
    x[1, 40] = bad
    kept = ra.ra_checkpoint8_pack(x)
    assert int(kept.e[1, 1]) == 255 and not bool(kept.q[1, 32:64].any())
    back = ra.ra_checkpoint8_unpack(kept)
    nan = torch.zeros(3, cols, dtype=torch.bool, device="cuda")
    nan[1, 32:64] = True
    assert torch.equal(torch.isnan(back), nan[:, :cols])
    assert bool(torch.isnan(ra.ra_checkpoint8_unpack(kept, act="gelu")[nan]).all())


@pytest.mark.parametrize("rows,cols", [(0, 8), (4, 0), (0, 0)])
def test_nothing_to_do(rows, cols):
    kept = ra.ra_checkpoint8_pack(torch.empty(rows, cols, device="cuda"))
    assert ra.ra_checkpoint8_unpack(kept).shape == (rows, cols)


def test_refusals():
    x = torch.zeros(4, 64, device="cuda")
    with pytest.raises(ValueError):
        ra.ra_checkpoint8_pack(torch.zeros(4, 64))
    with pytest.raises(TypeError):
        ra.ra_checkpoint8_pack(x.double())
    with pytest.raises(ValueError):
        ra.ra_checkpoint8_pack(x.t())
    with pytest.raises(ValueError):
        ra.ra_checkpoint8_pack(x, out=ra.Checkpoint8(4, 32))
    with pytest.raises(ValueError):
        ra.ra_checkpoint8_unpack(ra.Checkpoint8(4, 64), act="tanh")
    with pytest.raises(ValueError):
        ra.Checkpoint8(4, 64, q=torch.zeros(4, 60, dtype=torch.int8, device="cuda"), e=torch.zeros(4, 2, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        ra.Checkpoint8(4, 64, q=torch.zeros(4, 64, dtype=torch.int8, device="cuda"))
