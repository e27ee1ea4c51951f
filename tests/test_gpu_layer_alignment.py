"""A layer's bias at every alignment that its dtype allows, on the sizes that go to the large tiles, the ring and
the kernels for few rows."""
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


# (sizes, n, k, the kernel where every operand suits it)
SIZES = [([260, 300], 6200, 128, "grouped_256_nt"), ([700, 900], 520, 2560, "grouped_256_nt"),
         ([70, 40, 90], 512, 640, "grouped_ring_nt"), ([3, 0, 5], 96, 200, "grouped_rows_bf16")]


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("lead", [0, 1, 2, 3])
@pytest.mark.parametrize("i", range(len(SIZES)))
def test_bias_between_dwords(i, lead, residual):
    sizes, n, k, kernel = SIZES[i]
    bounds = grouped_ref.bounds_of(sizes, 1)
    rows, e = bounds[-1] + 2, len(sizes)
    off = torch.tensor(bounds, dtype=torch.int64, device="cuda")
    X, W = _rand((rows, k), 1), _rand((e, n, k), 2, 0.1)
    buf = torch.full((lead + e * n + 9,), float("nan"), dtype=BF, device="cuda")
    b = buf[lead:lead + e * n].view(e, n)
    b.copy_(_rand((e, n), 3))
    R = _rand((rows, n), 4) if residual else None
    print("case", sizes, n, k, lead, residual, flush=True)
    mns.profile_begin()
    try:
        Y, Z = mns.grouped_linear(X, W, off, bias=b, activation="gelu", residual=R, keep_z=True)
    finally:
        names = [r["name"] for r in mns.profile_end()]
    if lead % 2 == 0:
        assert names == [kernel]
    zero = torch.zeros(rows, n, dtype=BF)
    wY, eY, wZ, eZ = ref.linear(X, W, bounds, b, "gelu", R, zero, zero)
    grouped_ref.check(Y, wY, eY, "Y")
    grouped_ref.check(Z, wZ, eZ, "Z")
