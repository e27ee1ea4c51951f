"""The float64 gradient the GPU tests compare with, pinned against the closed form in the singular
basis, torch's automatic differentiation and differences of the forward map; and the refusals of
ns_orthogonalize_backward that need no GPU."""
import ctypes

import numpy as np
import pytest
import torch

import muon_newton_schulz_amd as mns
import ns_backward_ref as ref
import oracle
from muon_newton_schulz_amd import _abi

QUINTIC = (3.4445, -4.7750, 2.0315)
CONVERGENT = (15.0 / 8.0, -10.0 / 8.0, 3.0 / 8.0)
SHAPES = [(1, 1), (1, 7), (6, 6), (5, 12), (12, 5)]
COEFFS = {"quintic": [QUINTIC] * 5, "mixed": [QUINTIC] * 3 + [CONVERGENT] * 2,
          "cubic": [(1.5, -0.5, 0.0)] * 4, "one": [(2.0, -1.5, 0.5)]}


def _pair(shape, seed=0):
    g = np.random.default_rng(seed)
    return g.standard_normal(shape), g.standard_normal(shape)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("name", sorted(COEFFS))
def test_reference_gradient_four_ways(shape, name):
    coeffs = COEFFS[name]
    X, G = _pair(shape)
    np.testing.assert_allclose(ref.forward(X, coeffs), oracle.newton_schulz(X, coeffs),
                               rtol=1e-11, atol=1e-13)
    got = ref.gradient(X, G, coeffs)
    scale = np.linalg.norm(G) / np.linalg.norm(X) * 500.0     # largest growth of a direction
    np.testing.assert_allclose(got, ref.gradient_svd(X, G, coeffs), atol=1e-11 * scale, rtol=1e-8)
    x = torch.tensor(X, requires_grad=True)
    y = x / torch.linalg.norm(x)
    y = y.t() if shape[0] > shape[1] else y
    for a, b, c in coeffs:
        s = y @ y.t()
        y = a * y + (b * s + c * s @ s) @ y
    y = y.t() if shape[0] > shape[1] else y
    y.backward(torch.tensor(G))
    np.testing.assert_allclose(got, x.grad.numpy(), atol=1e-12 * scale, rtol=1e-9)
    # central differences in random directions: h^2 f''' / 6 with h = 1e-5 of the norm
    rng = np.random.default_rng(5)
    for _ in range(3):
        D = rng.standard_normal(shape)
        h = 1e-5 * np.linalg.norm(X) / np.linalg.norm(D)
        num = np.sum(G * (ref.forward(X + h * D, coeffs) - ref.forward(X - h * D, coeffs))) / (2 * h)
        assert abs(num - np.sum(got * D)) <= 1e-4 * scale * np.linalg.norm(D)


def test_derivative_is_symmetric():
    """<J D, G> = <D, J G>: what lets the gradient be carried forward."""
    X, G = _pair((6, 9))
    D = np.random.default_rng(9).standard_normal((6, 9))
    n = np.linalg.norm(X)
    h = 1e-6
    # derivative at X / ||X|| without the normalisation: project it out of both directions
    X0 = X / n
    D -= X0 * np.sum(X0 * D)
    G -= X0 * np.sum(X0 * G)
    C5 = [QUINTIC] * 5
    jd = (ref.forward(X0 + h * D, C5) - ref.forward(X0 - h * D, C5)) / (2 * h)
    jg = (ref.forward(X0 + h * G, C5) - ref.forward(X0 - h * G, C5)) / (2 * h)
    assert abs(np.sum(jd * G) - np.sum(jg * D)) <= 1e-6 * np.linalg.norm(jd) * np.linalg.norm(G)


def _call(lib, T=5, coeffs=QUINTIC, **kw):
    a = dict(X=0x10000, dO=0x20000, dX=0x30000, dtype=_abi.MNS_BF16, batch=1, rows=300, cols=700,
             ws=0x100000, wsb=1 << 40)
    a.update(kw)
    abc = (ctypes.c_float * (3 * max(T, 1)))(*(list(coeffs) * max(T, 1)))
    return lib.ns_orthogonalize_backward(a["X"], a["dO"], a["dX"], a["dtype"], a["batch"],
                                         a["rows"], a["cols"], T, abc, a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), _abi.MNS_ERR_DTYPE),
    (dict(batch=0), _abi.MNS_ERR_SHAPE),
    (dict(rows=0), _abi.MNS_ERR_SHAPE),
    (dict(cols=65537), _abi.MNS_ERR_SHAPE),
    (dict(rows=20000, cols=40000), _abi.MNS_ERR_SHAPE),      # twice the iterate: past 2 GiB
    (dict(X=None), _abi.MNS_ERR_NULL),
    (dict(dO=None), _abi.MNS_ERR_NULL),
    (dict(dX=None), _abi.MNS_ERR_NULL),
    (dict(T=0), _abi.MNS_ERR_PARAM),
    (dict(T=65), _abi.MNS_ERR_PARAM),
    (dict(coeffs=(float("nan"), 0.0, 0.0)), _abi.MNS_ERR_PARAM),
    (dict(T=12), _abi.MNS_ERR_PARAM),                        # 3.4445^12 > 2^20
    (dict(T=10, ws=None), _abi.MNS_ERR_WORKSPACE),           # 3.4445^10 < 2^20: runs
    (dict(T=12, dtype=_abi.MNS_F32, ws=None), _abi.MNS_ERR_WORKSPACE),
    (dict(T=64, dtype=_abi.MNS_F32), _abi.MNS_ERR_PARAM),    # 3.4445^64 > 1e30
    (dict(X=0x10004), _abi.MNS_ERR_PARAM),
    (dict(dX=0x30008), _abi.MNS_ERR_PARAM),
    (dict(ws=None), _abi.MNS_ERR_WORKSPACE),
    (dict(ws=0x100010), _abi.MNS_ERR_WORKSPACE),
    (dict(wsb=1000), _abi.MNS_ERR_WORKSPACE),
])
def test_library_refuses(kw, status):
    assert _call(mns.load(), **kw) == status


def test_workspace_query():
    lib = mns.load()
    out = ctypes.c_size_t(0)
    assert lib.mns_ns_backward_workspace_size(1, 1, 300, 700, ctypes.byref(out)) == 0
    assert out.value >= 4 * 2 * 512 * 768 * 2                # two [E; X] and their transposes
    assert lib.mns_ns_backward_workspace_size(1, 1, 300, 700, None) == _abi.MNS_ERR_NULL
    assert lib.mns_ns_backward_workspace_size(5, 1, 300, 700, ctypes.byref(out)) == _abi.MNS_ERR_DTYPE
    assert lib.mns_ns_backward_workspace_size(1, 0, 300, 700, ctypes.byref(out)) == _abi.MNS_ERR_SHAPE


def test_binding_refusals():
    X = torch.zeros(8, 16)
    C5 = [QUINTIC] * 5
    with pytest.raises(ValueError, match="GPU"):
        mns.ns_orthogonalize_backward(X, X.clone(), C5)
    for dO in (torch.zeros(16, 8), torch.zeros(8, 16, dtype=torch.bfloat16),
               torch.zeros(16, 8).t()):
        with pytest.raises(ValueError):
            mns.ns_orthogonalize_backward(X, dO, C5)
    with pytest.raises(TypeError):
        mns.ns_orthogonalize_backward(X.half(), X.half(), C5)
    with pytest.raises(ValueError, match="overlap"):
        mns.ns_orthogonalize_backward(X, X.clone(), C5, out=X)
    with pytest.raises(ValueError):
        mns.ns_orthogonalize_backward(X[0], X[0], C5)


@pytest.mark.parametrize("rows,cols", [(300, 570), (570, 300), (257, 560), (64, 4096), (16, 12288),
                                       (256, 256), (100, 700), (512, 512), (1024, 1024)])
def test_workspace_of_a_batch_covers_its_last_chunk(rows, cols):
    """Batches run in chunks of 32; a shorter last one may take another form, with buffers of
    other sizes, on the same workspace."""
    lib = mns.load()
    out = ctypes.c_size_t()
    for dtype in (_abi.MNS_F32, _abi.MNS_BF16):
        def size(batch):
            assert lib.mns_ns_backward_workspace_size(dtype, batch, rows, cols, ctypes.byref(out)) == 0
            return out.value
        for rest in range(1, 32):
            assert size(32 + rest) >= max(size(32), size(rest))
