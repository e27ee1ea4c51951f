"""Every form of a layer (activation, Z kept or not, bias or none, residual or none) on the kernels that the DMA
feeds: 256 x 256 tiles whole and cut into parts, and the ring; dense, and with row pitches wider than the rows
whose gaps and outside must stay as they are."""
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


# (sizes, width of the output, reduction), the kernels' name without its direction
SIZES = {"grouped_256": ([260, 300], 6200, 128), "grouped_ring": ([70, 40, 90], 512, 640),
         "parts": ([700, 900], 520, 2560)}


def _wide(t, gap):
    """t's values in rows `gap` elements wider, 16-byte aligned, in a buffer of 7s with a row before and behind."""
    buf = torch.full((t.shape[0] + 2, t.shape[1] + gap), 7.0, dtype=BF, device="cuda")
    view = buf[1:-1, 8:8 + t.shape[1]]
    view.copy_(t)
    return view, buf


def _only_the_view(buf, view, old):
    view.copy_(old)
    return (buf[0] == 7).all() and (buf[-1] == 7).all() and (buf[1:-1, :8] == 7).all() and (
        buf[1:-1, 8 + view.shape[1]:] == 7).all()


def _names(call):
    mns.profile_begin()
    try:
        out = call()
    finally:
        names = [r["name"] for r in mns.profile_end()]
    return out, names


FORMS = [(act, keep, residual) for act in [None] + ref.ACTS for keep in (False, True) for residual in (False, True)
         if act or not keep]


@pytest.mark.parametrize("pitched", [False, True], ids=["dense", "pitched"])
@pytest.mark.parametrize("kernel", sorted(SIZES))
@pytest.mark.parametrize("act,keep,residual", FORMS)
def test_forward(act, keep, residual, kernel, pitched):
    sizes, n, k = SIZES[kernel]
    bounds = grouped_ref.bounds_of(sizes, 1)
    rows, e = bounds[-1] + 2, len(sizes)
    off = torch.tensor(bounds, dtype=torch.int64, device="cuda")
    X, W = _rand((rows, k), 1), _rand((e, n, k), 2, 0.1)
    bias = _rand((e, n), 3) if residual != keep else None
    R = _rand((rows, n), 4) if residual else None
    zero = torch.zeros(rows, n, dtype=BF, device="cuda")
    old, oldz, args = zero, zero, {}
    if pitched:
        X = _wide(X, 8)[0]
        R = _wide(R, 16)[0] if residual else None
        old, oldz = _rand((rows, n), 5), _rand((rows, n), 6)
        out, buf = _wide(old, 24)
        oz, bufz = _wide(oldz, 40)
        args = {"out": out, "out_z": oz} if keep else {"out": out}
    print("case", act, keep, residual, kernel, pitched, flush=True)
    got, names = _names(lambda: mns.grouped_linear(X, W, off, bias=bias, activation=act, residual=R, keep_z=keep,
                                                   **args))
    assert names == [("grouped_256" if kernel == "parts" else kernel) + "_nt"]
    wY, eY, wZ, eZ = ref.linear(X, W, bounds, bias, act, R, old, oldz)
    if keep:
        got, Z = got
        grouped_ref.check(Z, wZ, eZ, "Z")
    grouped_ref.check(got, wY, eY, "Y")
    if pitched:
        assert _only_the_view(buf, out, old) and _only_the_view(bufz, oz, oldz)


@pytest.mark.parametrize("pitched", [False, True], ids=["dense", "pitched"])
@pytest.mark.parametrize("kernel", sorted(SIZES))
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("act", [None] + ref.ACTS)
def test_input_gradient(act, residual, kernel, pitched):
    sizes, k, n = SIZES[kernel]
    bounds = grouped_ref.bounds_of(sizes, 1)
    rows, e = bounds[-1] + 2, len(sizes)
    off = torch.tensor(bounds, dtype=torch.int64, device="cuda")
    dY, W = _rand((rows, n), 1), _rand((e, n, k), 2, 0.1)
    Z = _rand((rows, k), 3) if act else None
    R = _rand((rows, k), 4) if residual else None
    old, args = torch.zeros(rows, k, dtype=BF, device="cuda"), {}
    if pitched:
        dY = _wide(dY, 8)[0]
        Z = _wide(Z, 40)[0] if act else None
        R = _wide(R, 16)[0] if residual else None
        old = _rand((rows, k), 5)
        out, buf = _wide(old, 24)
        args = {"out": out}
    print("case", act, residual, kernel, pitched, flush=True)
    got, names = _names(lambda: mns.grouped_input_grad(dY, W, off, activation=act, Z=Z, residual=R, **args))
    assert names == [("grouped_256" if kernel == "parts" else kernel) + "_nn"]
    grouped_ref.check(got, *ref.input_grad(dY, W, bounds, act, Z, R, old), "dX")
    if pitched and (residual or act):                                     # in place, over an operand
        same, _ = _wide(R if residual else Z, 24)
        mns.grouped_input_grad(dY, W, off, activation=act, Z=Z if residual else same,
                               residual=same if residual else None, out=same)
        assert torch.equal(same[bounds[0]:bounds[-1]], got[bounds[0]:bounds[-1]])
    if pitched:
        assert _only_the_view(buf, out, old)
