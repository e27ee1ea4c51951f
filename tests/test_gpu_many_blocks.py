"""Calls of more tiles than a row of a launch's grid holds: 2^21, and at most 2^32 threads."""
import pytest
import torch

import muon_newton_schulz_amd as mns

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
MOST = 65536


@pytest.fixture(autouse=True)
def _room():
    if torch.cuda.mem_get_info()[0] < 32 << 30:
        pytest.skip("needs 32 GB of GPU memory")
    yield
    torch.cuda.empty_cache()


def _one_each(experts):
    return torch.arange(experts + 1, dtype=torch.int64, device="cuda")


def _normal(shape, seed):
    return torch.empty(shape, dtype=BF, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(seed))


def test_bias_gradient():
    """16385 experts x 65536 columns: 2^22 + 8704 blocks, then 2^22 + 256 of 1024 threads that join."""
    rows, experts = 1000, MOST // 4 + 1
    owners = {3: (0, 300), 10000: (300, 301), experts - 1: (301, 1000)}
    off = torch.zeros(experts + 1, dtype=torch.int64)
    for e, (_, hi) in owners.items():
        off[e + 1:] = hi
    dY = _normal((rows, MOST), 1)
    print("case bias gradient", flush=True)
    db = mns.grouped_bias_grad(dY, off.cuda())
    for e, (lo, hi) in owners.items():
        part = dY[lo:hi].double()
        err = (hi - lo + 2) * 2.0 ** -23 * part.abs().sum(0)
        want = part.sum(0)
        assert ((db[e].double() - want).abs() <= err + 2.0 ** -8 * (want.abs() + err)).all(), e
        db[e] = 0
    assert all(not chunk.any() for chunk in db.split(4096))


def test_layer():
    """One row each for 16384 experts of 65536 x 1: 2^22 + 2^18 tiles of 16 x 256."""
    rows = MOST // 4
    X, W, off = _normal((rows, 1), 2), _normal((rows, MOST, 1), 3), _one_each(rows)
    for name, call in (("linear", lambda: mns.grouped_linear(X, W, off)),
                       ("matmul", lambda: mns.grouped_matmul(X, W, off))):
        print("case", name, flush=True)
        Y = call()
        for i in range(0, rows, 4096):
            part = slice(i, i + 4096)
            assert torch.equal(Y[part], (X[part].float() * W[part, :, 0].float()).to(BF)), (name, i)
        del Y


def test_weight_gradient():
    """65536 experts of 1 x 65536: 2^25 tiles of 128 x 128."""
    dY, X = _normal((MOST, 1), 4), _normal((MOST, MOST), 5)
    print("case weight gradient", flush=True)
    G = mns.grouped_weight_grad(dY, X, _one_each(MOST))
    for i in range(0, MOST, 4096):
        part = slice(i, i + 4096)
        assert torch.equal(G[part, 0], (dY[part].float() * X[part].float()).to(BF)), i
