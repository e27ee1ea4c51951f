"""Bias gradients of more experts than a wave holds, several chunks long on either side of the 64th, and offsets
that are not what they should be, whose outputs lie between guards."""
import pytest
import torch

import grouped_ref
import layer_ref as ref
import muon_newton_schulz_amd as mns

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _rand(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype).cuda()


# experts with more rows than a chunk (32 and up), the others have 0 to 4
LONG = {70: {0: 300, 62: 100, 63: 129, 64: 200, 65: 90, 69: 400},
        150: {1: 65, 63: 70, 64: 33, 127: 600, 128: 257, 129: 40, 149: 500}}


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("front,tail", [(0, 0), (5, 0), (130, 70)])
@pytest.mark.parametrize("experts", sorted(LONG))
def test_bias_gradient_of_many_experts(experts, front, tail, dtype):
    sizes = [LONG[experts].get(e, (e * 7) % 5) for e in range(experts)]
    bounds = grouped_ref.bounds_of(sizes, front)
    rows, n = bounds[-1] + tail, 600
    off = torch.tensor(bounds, dtype=torch.int64, device="cuda")
    dY, Z = _rand((rows, n), dtype, 1), _rand((rows, n), dtype, 2)
    print("case", experts, front, tail, dtype, flush=True)
    db, dZ = mns.grouped_bias_grad(dY, off, activation="silu", Z=Z, out_dtype=F32)
    wb, eb, wz, ez = ref.bias_grad(dY, bounds, "silu", Z, F32, torch.zeros(rows, n))
    grouped_ref.check(db, wb, eb, "db")
    grouped_ref.check(dZ, wz, ez, "dZ")
    kept = _rand((rows, n), dtype, 3)                  # a given dZ keeps the rows of no expert
    out = kept.clone()
    db2, _ = mns.grouped_bias_grad(dY, off, activation="silu", Z=Z, out_dtype=F32, out_dz=out)
    assert torch.equal(db2, db) and torch.equal(out[bounds[0]:bounds[-1]], dZ[bounds[0]:bounds[-1]])
    assert torch.equal(out[:front], kept[:front]) and torch.equal(out[bounds[-1]:], kept[bounds[-1]:])
    plain = mns.grouped_bias_grad(dY, off, out_dtype=F32)
    wb, eb, _, _ = ref.bias_grad(dY, bounds, None, None, F32, torch.zeros(rows, n))
    grouped_ref.check(plain, wb, eb, "no activation")


def _between(rows, width, dtype, gap):
    """A view of rows x width, its buffer of 7s, and the view's place in it."""
    buf = torch.full((rows + 16, width + gap), 7.0, dtype=dtype, device="cuda")
    return buf[8:8 + rows, :width], buf


def _guards(buf, rows, width):
    return (buf[:8] == 7).all() and (buf[8 + rows:] == 7).all() and (buf[:, width:] == 7).all()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,n,k", [(900, 512, 256), (90, 70, 2100), (40, 96, 72), (700, 6200, 128)])
@pytest.mark.parametrize("bounds", [[0, 0.9, 0, 0.9, 0], [-5, 2 ** 40, 7, -(2 ** 50), 3], [1, 1, 0, 0, 1],
                                    [0, 1, 0, 1, 1]], ids=["overlap", "outside", "backwards", "twice"])
def test_wrong_offsets_write_nothing_outside(bounds, rows, n, k, dtype):
    """Values are unspecified; a fraction stands for that part of the rows."""
    off = torch.tensor([int(b * rows) if isinstance(b, float) or b == 1 else b for b in bounds],
                       dtype=torch.int64, device="cuda")
    e = len(bounds) - 1
    W, b = _rand((e, n, k), dtype, 1, 0.1), _rand((e, n), dtype, 2)
    X, dY, Z = _rand((rows, k), dtype, 3), _rand((rows, n), dtype, 4), _rand((rows, k), dtype, 5)
    print("case", bounds, rows, n, k, dtype, flush=True)
    (y, by), (z, bz) = _between(rows, n, dtype, 8), _between(rows, n, dtype, 24)
    mns.grouped_linear(X, W, off, bias=b, activation="gelu", residual=dY, out=y, out_z=z)
    assert _guards(by, rows, n) and _guards(bz, rows, n)
    x, bx = _between(rows, k, dtype, 8)
    mns.grouped_input_grad(dY, W, off, activation="gelu", Z=Z, out=x)
    assert _guards(bx, rows, k)
    x, bx = _between(rows, k, dtype, 3)
    db, bd = _between(e, k, F32, 0)
    mns.grouped_bias_grad(X, off, activation="gelu", Z=Z, out=db, out_dz=x)
    assert _guards(bx, rows, k) and _guards(bd, e, k)
    bg = torch.full((e + 2, n, k), 7.0, dtype=F32, device="cuda")
    mns.grouped_weight_grad(dY, X, off, out=bg[1:-1], out_dtype=F32)
    assert (bg[0] == 7).all() and (bg[-1] == 7).all()
