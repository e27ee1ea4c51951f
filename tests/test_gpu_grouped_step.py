"""muon_step_grouped against the float64 step on the gradients its tokens stand for, and a training
round of a layer of experts with orthogonalised weights, through every operator it takes: forward,
input gradient, weight gradient, the Newton-Schulz gradient and the step."""
import numpy as np
import pytest
import torch

import grouped_ref
import muon_newton_schulz_amd as mns
import ns_backward_ref
import oracle
from helpers import TOL, check_weight, rel, to_f64

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
QUINTIC = (3.4445, -4.7750, 2.0315)
C5 = [QUINTIC] * 5


def _rand(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype).cuda()


CASES = [
    # dtype, sizes, rows, cols, kind, normuon
    (BF, [70, 0, 130, 9], 96, 160, "standard", False),
    (BF, [70, 0, 130, 9], 96, 160, "gram", True),
    (BF, [33, 64], 300, 270, "standard", True),
    (F32, [5, 40, 0], 33, 65, "standard", False),
    (F32, [64, 1], 130, 70, "gram", True),
    (BF, [3] * 35, 24, 40, "standard", True),          # more than one chunk of matrices
]


@pytest.mark.parametrize("dtype,sizes,rows,cols,kind,normuon", CASES)
def test_step_from_tokens(dtype, sizes, rows, cols, kind, normuon):
    storage = "bf16" if dtype == BF else "f32"
    bounds = grouped_ref.bounds_of(sizes, 2)
    total, e = bounds[-1] + 3, len(sizes)
    W = _rand((e, rows, cols), dtype, 1, 0.05)
    M = _rand((e, rows, cols), F32, 2, 0.5)
    v = torch.rand(e, rows, generator=torch.Generator().manual_seed(3)).cuda() if normuon else None
    dY, X = _rand((total, rows), dtype, 4), _rand((total, cols), dtype, 5)
    off = torch.tensor(bounds, device="cuda")
    restart = (3,) if kind == "gram" else ()
    W0, M0 = to_f64(W), to_f64(M)
    v0 = to_f64(v) if normuon else None
    want_m, err_m = grouped_ref.weight_grad(dY, X, bounds, M, 0.9, F32)
    mns.muon_step_grouped(W, M, dY, X, off, v, mu=0.9, lr=0.02, coeffs=C5, kind=kind,
                          restart_before=restart, normuon=normuon)
    grouped_ref.check(M, want_m, err_m, "momentum")
    dYd, Xd = to_f64(dY), to_f64(X)
    for i, (lo, hi) in enumerate(zip(bounds, bounds[1:])):
        G = dYd[lo:hi].T @ Xd[lo:hi]
        out = oracle.muon_step(W0[i], M0[i], G, mu=0.9, lr=0.02, coeffs=C5, kind=kind,
                               restart_before=restart, normuon=normuon,
                               v=v0[i] if normuon else None, beta2=0.95, eps=1e-8)
        check_weight(to_f64(W[i]), W0[i], out["W_exact"] - W0[i], storage, f"W[{i}]")
        if normuon:
            assert rel(to_f64(v[i]), out["v"]) <= TOL[storage]


def test_equals_the_step_on_formed_gradients_in_float32():
    """With float32 storage the formed gradient is unrounded too: the two steps differ by the order
    and number of roundings of mu M + G, a few units of 2^-24, far inside the parity gate."""
    sizes, rows, cols = [40, 25], 48, 96
    bounds = grouped_ref.bounds_of(sizes)
    off = torch.tensor(bounds, device="cuda")
    dY, X = _rand((65, rows), F32, 1), _rand((65, cols), F32, 2)
    W, M = _rand((2, rows, cols), F32, 3, 0.1), _rand((2, rows, cols), F32, 4)
    G = mns.grouped_weight_grad(dY, X, off)
    W2, M2 = W.clone(), M.clone()
    mns.muon_step([W2[0], W2[1]], [M2[0], M2[1]], [G[0], G[1]], mu=0.9, lr=0.02, coeffs=C5)
    W1, M1 = W.clone(), M.clone()
    mns.muon_step_grouped(W1, M1, dY, X, off, mu=0.9, lr=0.02, coeffs=C5)
    for i in range(2):
        assert rel(to_f64(M1[i]), to_f64(M2[i])) <= 1e-6
        assert rel(to_f64(W1[i] - W[i]), to_f64(W2[i] - W[i])) <= TOL["f32"]


def test_step_captured_and_replayed():
    sizes, rows, cols = [50, 0, 70], 64, 200
    off = torch.tensor(grouped_ref.bounds_of(sizes), device="cuda")
    dY, X = _rand((120, rows), BF, 1), _rand((120, cols), BF, 2)
    W, M = _rand((3, rows, cols), BF, 3, 0.1), _rand((3, rows, cols), F32, 4)
    args = dict(mu=0.9, lr=0.02, coeffs=C5)
    ws = torch.empty(mns.grouped_step_workspace_size(W, M, dY, X, off, coeffs=C5),
                     dtype=torch.uint8, device="cuda")
    W2, M2 = W.clone(), M.clone()
    mns.muon_step_grouped(W2.clone(), M2.clone(), dY, X, off, workspace=ws, **args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mns.muon_step_grouped(W, M, dY, X, off, workspace=ws, **args)
    for i in range(3):
        dY.copy_(_rand((120, rows), BF, 10 + i))
        mns.muon_step_grouped(W2, M2, dY, X, off, **args)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(W, W2) and torch.equal(M, M2), i


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_training_round_of_orthogonalised_experts(dtype):
    """W_e = NS(V_e), Y = X W_e^T, L = <dY, Y>: the layer's gradients through the four operators
    against float64, and differences of the loss in float64; then the step on V."""
    storage = "bf16" if dtype == BF else "f32"
    sizes, n, k = [60, 0, 41, 7], 80, 144
    bounds = grouped_ref.bounds_of(sizes)
    total, e = bounds[-1] + 2, len(sizes)
    off = torch.tensor(bounds, device="cuda")
    V = _rand((e, n, k), dtype, 1)
    X, dY = _rand((total, k), dtype, 2), _rand((total, n), dtype, 3)

    W = mns.ns_orthogonalize(V, C5)
    Y = mns.grouped_matmul(X, W, off)
    dX = mns.grouped_matmul(dY, W, off, transpose_w=True)
    dW = mns.grouped_weight_grad(dY, X, off)
    dV = mns.ns_orthogonalize_backward(V, dW, C5)

    # each operator against float64 on the inputs it was given
    zeros = torch.zeros_like
    grouped_ref.check(Y, *grouped_ref.matmul(X, W, bounds, False, zeros(Y)), "Y")
    grouped_ref.check(dX, *grouped_ref.matmul(dY, W, bounds, True, zeros(dX)), "dX")
    grouped_ref.check(dW, *grouped_ref.weight_grad(dY, X, bounds, None, 0.0, dtype), "dW")
    Vd, Xd, dYd, dWd = to_f64(V), to_f64(X), to_f64(dY), to_f64(dW)
    loss = lambda Vs: sum(np.sum(dYd[lo:hi] * (Xd[lo:hi] @ ns_backward_ref.forward(Vs[i], C5).T))
                          for i, (lo, hi) in enumerate(zip(bounds, bounds[1:])))
    exact_dV = np.zeros_like(Vd)
    for i, (lo, hi) in enumerate(zip(bounds, bounds[1:])):
        assert rel(to_f64(W[i]), ns_backward_ref.forward(Vd[i], C5)) <= TOL[storage]
        if lo == hi:
            assert not dW[i].any() and not dV[i].any()
            continue
        exact_dW = dYd[lo:hi].T @ Xd[lo:hi]
        exact_dV[i] = ns_backward_ref.gradient(Vd[i], exact_dW, C5)
        # the whole chain: the last operator's gate, plus what dW's rounding becomes in it
        through = ns_backward_ref.gradient(Vd[i], dWd[i], C5)
        room = (TOL[storage] * np.linalg.norm(through)
                + np.linalg.norm(ns_backward_ref.gradient(Vd[i], dWd[i] - exact_dW, C5)))
        assert np.linalg.norm(to_f64(dV[i]) - exact_dV[i]) <= room
    # and the float64 chain against differences of the loss: a step of 1e-5 in entries of size 1
    # leaves a truncation below 1e-3 of the largest value the derivative can take
    D = np.random.default_rng(0).standard_normal(Vd.shape)
    h = 1e-5
    num = (loss(Vd + h * D) - loss(Vd - h * D)) / (2 * h)
    assert abs(num - np.sum(exact_dV * D)) <= 1e-3 * np.linalg.norm(exact_dV) * np.linalg.norm(D)

    M = torch.zeros(e, n, k, device="cuda")
    V0 = to_f64(V)
    mns.muon_step([V[i] for i in range(e)], [M[i] for i in range(e)], [dV[i] for i in range(e)],
                  mu=0.9, lr=0.02, coeffs=C5)
    assert torch.equal(V[1].cpu().double(), torch.from_numpy(V0[1]))     # no rows, no update
    for i in (0, 2, 3):
        assert not np.array_equal(to_f64(V[i]), V0[i])
