"""Rows, gradients and lists whose elements lie more than 2^31 apart: pitched operands against the same call on
dense ones, bit for bit."""
import pytest
import torch

import muon_newton_schulz_amd as mns

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
PITCH = 1 << 17


@pytest.fixture(autouse=True)
def _room():
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 100 GB of GPU memory")
    yield
    torch.cuda.empty_cache()


def _rand(shape, dtype, seed, scale=1.0):
    g = torch.Generator("cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _far(t):
    """t's values in rows 2^17 elements apart."""
    buf = torch.zeros(t.shape[0] * PITCH + t.shape[1], dtype=t.dtype, device="cuda")
    view = buf.as_strided(t.shape, (PITCH, 1))
    view.copy_(t)
    return view


# sizes that go to the large tiles, the ring, 128 x 128 and 64 x 64 tiles and the kernels for few rows
@pytest.mark.parametrize("dtype,experts,n,k", [(BF, 3, 512, 256), (BF, 150, 1024, 128), (BF, 3, 515, 130),
                                               (F32, 3, 72, 40), (BF, 400, 100, 36)])
def test_layers(dtype, experts, n, k):
    rows = 20000
    off = torch.linspace(0, rows, experts + 1).long().cuda()
    W, b = _rand((experts, n, k), dtype, 1, 0.1), _rand((experts, n), dtype, 2)
    X, R, dY = _rand((rows, k), dtype, 3), _rand((rows, n), dtype, 4), _rand((rows, n), dtype, 5)
    Z = _rand((rows, k), dtype, 6)
    print("case", dtype, experts, n, k, flush=True)
    want = mns.grouped_linear(X, W, off, bias=b, activation="silu", residual=R, keep_z=True)
    out, oz = _far(R), _far(R)
    mns.grouped_linear(_far(X), W, off, bias=b, activation="silu", residual=out, out=out, out_z=oz)
    assert torch.equal(out, want[0]) and torch.equal(oz, want[1])
    del out, oz
    want = mns.grouped_input_grad(dY, W, off, activation="gelu", Z=Z, residual=X)
    far = _far(Z)
    mns.grouped_input_grad(_far(dY), W, off, activation="gelu", Z=far, residual=_far(X), out=far)
    assert torch.equal(far, want)
    del far
    want = mns.grouped_bias_grad(dY, off, activation="gelu", Z=R)
    got = mns.grouped_bias_grad(_far(dY), off, activation="gelu", Z=_far(R), out_dz=_far(dY))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_balance():
    tokens, experts = 20000, 72
    ids = torch.randint(-1, experts, (tokens, 3), device="cuda")
    counts, _, _ = mns.expert_order(ids, experts)
    logits = _rand((tokens, experts), F32, 1)
    want = mns.balance_loss(logits, ids, counts)
    far = _far(logits)
    got = mns.balance_loss(far, ids, counts, out=far)
    assert torch.equal(got[0], want[0]) and torch.equal(far, want[1])


@pytest.mark.parametrize("dtype,lead", [(BF, 0), (F32, 1)], ids=["bf16", "f32"])
def test_clip(dtype, lead):
    """A gradient of 2^32 + 4101 elements, with a small one behind it."""
    n = (1 << 32) + 4101
    buf = torch.zeros(n + 100, dtype=dtype, device="cuda")
    grads = [buf[lead:lead + n], buf[lead + n + 7:lead + n + 57]]
    marks = [0, (1 << 31) - 1, 1 << 31, (1 << 32) - 1, 1 << 32, n - 1]
    for i, at in enumerate(marks):
        grads[0][at] = float(i + 1)
    grads[1][:] = 2.0
    norm = (sum((i + 1) ** 2 for i in range(len(marks))) + 50 * 4) ** 0.5
    got = mns.clip_grad_norm(grads, norm / 2, eps=0.0)
    assert abs(got.item() - norm) <= 2.0 ** -24 * norm + 1e-10
    # max_norm as float32, the factor and the product are rounded once each; bfloat16's steps hide that here
    off = 3 * 2.0 ** -24 if dtype == F32 else 0.0
    assert all(abs(grads[0][at].item() - (i + 1) / 2) <= off * (i + 1) / 2 for i, at in enumerate(marks))
    assert ((grads[1] - 1).abs() <= off).all() and not buf[lead + n:lead + n + 7].any()
    assert sum(int(p.count_nonzero()) for p in grads[0].split(1 << 30)) == len(marks)
