"""What the activations of bfloat16 layers and their slopes are before they are rounded: the slope as a bias
gradient of one row an expert in float32, the value with its own rounding taken away by the residual. Against
float64, at every bfloat16 number from 2^-20 to 13.25."""
import math

import pytest
import torch

import layer_ref as ref
import muon_newton_schulz_amd as mns

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
ULP = 2.0 ** -23


def _numbers():
    """(rows, 64) of them, both signs."""
    bits = torch.arange(0x3580, 0x4155, dtype=torch.int32)
    z = torch.cat([bits, bits + 0x8000])
    z = torch.cat([z, torch.zeros(-len(z) % 64, dtype=torch.int32)])
    return (z << 16).view(F32).to(BF).reshape(-1, 64)


def _errors(name, z):
    """Largest errors of the float32 value and slope. gelu: the fit of Q (1.5e-5 of it up to 5, 2.1e-4 up to 8,
    2.8e-3 beyond) and nine roundings of its logarithm, up to z^2 / 2 + 8; the slope's fit, 1.3e-6, and 16
    roundings, the exponential's argument rounded to z^2 2^-24. silu: sigmoid's argument and four roundings;
    1 - s is off by as much as s, and by its own rounding. Anything below 2^-126 may be flushed."""
    a = z.abs()
    value, slope, _ = ref.act(name, z)
    flush = 2.0 ** -126 * (1 + a)
    if name == "gelu":
        q, phi = 0.5 * torch.erfc(a / math.sqrt(2)), torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        fit = torch.where(a <= 5, 1.5e-5, torch.where(a <= 8, 2.1e-4, 2.8e-3)) + 9 * (z * z / 2 + 8) * ULP / 2
        return (a * q * fit + value.abs() * ULP + flush,
                (q + a * phi) * (1.3e-6 + (z * z + 16) * ULP) + slope.abs() * ULP + flush)
    s = torch.sigmoid(z)
    rel = (a + 4) * ULP
    return (value.abs() * (rel + ULP) + flush,
            s * ((1 + a * (1 - s)) * (rel + 3 * ULP) + a * (s * rel + ULP)) + flush)


@pytest.mark.parametrize("name", ["gelu", "silu"])
def test_slope(name):
    z = _numbers()
    rows = z.shape[0]
    off = torch.arange(rows + 1, dtype=torch.int64, device="cuda")
    db, _ = mns.grouped_bias_grad(torch.ones(rows, 64, dtype=BF, device="cuda"), off, activation=name,
                                  Z=z.cuda(), out_dtype=F32)
    want, err = ref.act(name, z.double())[1], _errors(name, z.double())[1]
    over = (db.cpu().double() - want).abs() / err
    assert over.max() <= 1, (name, over.max().item(), z.reshape(-1)[over.argmax()].item())


@pytest.mark.parametrize("name", ["gelu", "silu"])
def test_value(name):
    """act(z) - r, r the bfloat16 number next to it: the difference is exact, its rounding 2^-8 of it."""
    z = _numbers()
    want = ref.act(name, z.double())[0]
    r = want.to(BF)
    off = torch.tensor([0, z.shape[0]], dtype=torch.int64, device="cuda")
    W = torch.eye(64, dtype=BF, device="cuda")[None].contiguous()
    got = mns.grouped_linear(z.cuda(), W, off, activation=name, residual=-r.cuda())
    rest = want - r.double()
    err = _errors(name, z.double())[0]
    over = (got.cpu().double() - rest).abs() / (err + 2.0 ** -8 * (rest.abs() + err))
    assert over.max() <= 1, (name, over.max().item(), z.reshape(-1)[over.argmax()].item())
