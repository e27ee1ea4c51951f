"""Layers on the 256 x 256 kernel whose tiles end early: experts of 1 to 255 rows behind whole tiles, a last column
tile of 8 to 248, with the operands' last rows at the end of their buffers and NaN between the experts'."""
import pytest
import torch

import grouped_ref
import layer_ref as ref
import muon_newton_schulz_amd as mns

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _rand(shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(BF).cuda()


@pytest.mark.parametrize("last", [1, 9, 31, 32, 33, 127, 129, 255])
@pytest.mark.parametrize("width", [6152, 6392])
def test_part_tiles(last, width):
    sizes = [256 + last, 511 - last]
    bounds = grouped_ref.bounds_of(sizes, 1)
    rows, e, red = bounds[-1], len(sizes), 128
    off = torch.tensor(bounds, dtype=torch.int64, device="cuda")
    zero = torch.zeros(rows, width, dtype=BF)
    A, b = _rand((rows, red), 1), _rand((e, width), 3)
    R, Z = _rand((rows, width), 4), _rand((rows, width), 5)
    for t in (A, R, Z):
        t[:1] = float("nan")                       # a row of no expert
    W = _rand((e, width, red), 2, 0.1)
    print("case", sizes, width, "forward", flush=True)
    mns.profile_begin()
    got = mns.grouped_linear(A, W, off, bias=b, activation="silu", residual=R)
    plain = mns.grouped_linear(A, W, off, activation="relu")
    W2 = W.transpose(1, 2).contiguous()
    print("case", sizes, width, "input gradient", flush=True)
    back = mns.grouped_input_grad(A, W2, off, activation="gelu", Z=Z, residual=R)
    only = mns.grouped_input_grad(A, W2, off, residual=R)
    assert [r["name"] for r in mns.profile_end()] == ["grouped_256_nt", "grouped_256_nn"]
    wY, eY, _, _ = ref.linear(A, W, bounds, b, "silu", R, zero, zero)
    grouped_ref.check(got, wY, eY, "forward")
    wY, eY, _, _ = ref.linear(A, W, bounds, None, "relu", None, zero, zero)
    grouped_ref.check(plain, wY, eY, "forward, no bias")
    grouped_ref.check(back, *ref.input_grad(A, W2, bounds, "gelu", Z, R, zero), "input gradient")
    grouped_ref.check(only, *ref.input_grad(A, W2, bounds, None, None, R, zero), "residual only")
