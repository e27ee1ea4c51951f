"""ns_orthogonalize_backward against the float64 gradient, to the framework's parity gates (relative
Frobenius error per matrix: 1e-4 for float32 storage, 2e-2 for bfloat16), at sizes on both sides
of the padding, tile and arithmetic boundaries, and against differences of the GPU's own forward
map."""
import numpy as np
import pytest
import torch

import muon_newton_schulz_amd as mns
import ns_backward_ref as ref
import synthetic
from helpers import TOL, rel, stored_f64, to_device, to_f64

pytestmark = pytest.mark.gpu

QUINTIC = (3.4445, -4.7750, 2.0315)
CONVERGENT = (15.0 / 8.0, -10.0 / 8.0, 3.0 / 8.0)
C5 = [QUINTIC] * 5


def _say(*a):
    print(*a, flush=True)


def _batch(dist, batch, rows, cols, storage, tag):
    x = [synthetic.gradient(dist, rows, cols, storage, tag, 0, i) for i in range(batch)]
    g = [synthetic.gradient("normal", rows, cols, storage, tag, 1, i) for i in range(batch)]
    X = torch.stack([to_device(a, storage) for a in x])
    G = torch.stack([to_device(a, storage) for a in g])
    return X, G, [stored_f64(a, storage) for a in x], [stored_f64(a, storage) for a in g]


CASES = [
    ("f32", "normal", 1, 1, 1), ("f32", "normal", 3, 1, 9), ("f32", "student_t", 2, 100, 257),
    ("f32", "normal", 1, 256, 1024), ("f32", "lowrank", 1, 300, 200), ("f32", "normal", 1, 257, 257),
    ("bf16", "normal", 2, 1, 1), ("bf16", "normal", 5, 17, 23), ("bf16", "lowrank", 2, 64, 64),
    ("bf16", "lowrank", 1, 256, 256), ("bf16", "lowrank", 2, 257, 300), ("bf16", "student_t", 3, 1111, 333),
    ("bf16", "normal", 1, 512, 2048), ("bf16", "lowrank", 1, 700, 700), ("bf16", "normal", 40, 24, 130),
    ("f32", "normal", 3, 64, 64), ("f32", "student_t", 2, 64, 65), ("f32", "normal", 2, 3000, 33),
    ("bf16", "normal", 1, 63, 5000), ("bf16", "student_t", 33, 40, 96), ("bf16", "normal", 2, 129, 64),
    ("f32", "normal", 1, 65, 64), ("f32", "normal", 1, 65, 66),
    ("bf16", "student_t", 2, 1100, 2300), ("bf16", "normal", 1, 2300, 1100), ("f32", "normal", 35, 30, 20),
]


@pytest.mark.parametrize("storage,dist,batch,rows,cols", CASES)
def test_gradient(storage, dist, batch, rows, cols):
    _say("case", storage, dist, batch, rows, cols)
    if dist == "lowrank" and min(rows, cols) < 64:
        dist = "normal"
    X, G, xs, gs = _batch(dist, batch, rows, cols, storage, 31)
    dX = mns.ns_orthogonalize_backward(X, G, C5)
    for i in range(0, batch, max(1, batch // 4)):
        want = ref.gradient(xs[i], gs[i], C5)
        if min(rows, cols) == 1:
            # one singular value: the map is constant along X, and of the rest f(1)/1 remains;
            # a 1 x 1 gradient is zero, left with the rounding of its two terms
            scale = np.linalg.norm(gs[i]) / np.linalg.norm(xs[i])
            err = np.linalg.norm(to_f64(dX[i]) - want) / scale
        else:
            err = rel(to_f64(dX[i]), want)
        _say("  matrix", i, "error", f"{err:.2e}")
        assert err <= TOL[storage]


@pytest.mark.parametrize("storage", ["f32", "bf16"])
@pytest.mark.parametrize("coeffs", [[(1.5, -0.5, 0.0)] * 4, [QUINTIC] * 4 + [CONVERGENT] * 2,
                                    [(2.0, -1.5, 0.5)], [QUINTIC] * 10],
                         ids=["cubic", "mixed", "one", "ten"])
def test_coefficients(storage, coeffs):
    for rows, cols in ((300, 500), (400, 270)):
        X, G, xs, gs = _batch("normal", 1, rows, cols, storage, 7)
        dX = mns.ns_orthogonalize_backward(X[0], G[0], coeffs)
        err = rel(to_f64(dX), ref.gradient(xs[0], gs[0], coeffs))
        _say("case", storage, rows, cols, len(coeffs), f"error {err:.2e}")
        assert err <= TOL[storage]


def test_against_differences_of_the_forward_call():
    """<dX, D> against central differences of <G, ns_orthogonalize(X + h D)> on the GPU, float32.

    The difference's error: rounding of two float32 orthogonalisations (each within 1e-4 of the
    float64 one, the parity gate, but their errors mostly cancel) and the h^2 term. With h = 0.02
    of ||X|| both stay below 2 % of the largest value the derivative can take here."""
    X, G, xs, gs = _batch("normal", 1, 96, 320, "f32", 3)
    X, G = X[0], G[0]
    dX = mns.ns_orthogonalize_backward(X, G, [(1.5, -0.5, 0.0)] * 3).double()
    for seed in range(4):
        D = torch.randn(X.shape, generator=torch.Generator().manual_seed(seed)).cuda()
        # a direction with a clear derivative: half of it along the gradient
        D = D / D.norm() + (dX / dX.norm()).float()
        h = 0.02 * float(X.norm() / D.norm())
        lo, hi = (mns.ns_orthogonalize((X + s * h * D).contiguous(), [(1.5, -0.5, 0.0)] * 3).double()
                  for s in (-1.0, 1.0))
        num = float((G.double() * (hi - lo)).sum() / (2 * h))
        ana = float((dX * D.double()).sum())
        _say("direction", seed, num, ana)
        assert abs(num - ana) <= 0.02 * float(dX.norm() * D.double().norm())


@pytest.mark.parametrize("storage", ["f32", "bf16"])
def test_zero_tiny_and_huge(storage):
    """A zero input or gradient gives zeros; norms near the ends of the float32 range neither
    overflow nor vanish."""
    for rows, cols in ((70, 90), (300, 280)):
        X, G, xs, gs = _batch("normal", 4, rows, cols, storage, 11)
        X[0].zero_()
        G[1].zero_()
        X[2] *= 2.0 ** 100
        G[2] *= 2.0 ** 100          # dX of the unscaled size
        X[3] *= 2.0 ** -100
        G[3] *= 2.0 ** -100
        dX = mns.ns_orthogonalize_backward(X, G, C5)
        assert not dX[0].any() and not dX[1].any()
        for i in (2, 3):
            assert rel(to_f64(dX[i]), ref.gradient(xs[i], gs[i], C5)) <= TOL[storage]


def test_nonfinite_stays_in_its_matrix():
    X, G, xs, gs = _batch("normal", 3, 300, 400, "bf16", 13)
    clean = mns.ns_orthogonalize_backward(X, G, C5)
    X[0, 5, 7] = float("nan")
    G[2, 1, 1] = float("inf")
    dX = mns.ns_orthogonalize_backward(X, G, C5)
    assert torch.equal(dX[1], clean[1])
    assert not torch.isfinite(dX[0]).any() and not torch.isfinite(dX[2]).all()


def test_given_output_and_workspace_twice_the_same():
    X, G, _, _ = _batch("student_t", 2, 333, 555, "bf16", 17)
    need = mns.ns_backward_workspace_size(X)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")     # NaN patterns
    out = torch.empty_like(X)
    assert mns.ns_orthogonalize_backward(X, G, C5, out=out, workspace=ws) is out
    again = mns.ns_orthogonalize_backward(X, G, C5, workspace=ws)
    fresh = mns.ns_orthogonalize_backward(X, G, C5)
    assert torch.equal(out, again) and torch.equal(out, fresh)


def test_captured_and_replayed():
    X, G, _, _ = _batch("normal", 2, 200, 520, "bf16", 19)
    ws = torch.empty(mns.ns_backward_workspace_size(X), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(X)
    mns.ns_orthogonalize_backward(X, G, C5, out=out, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mns.ns_orthogonalize_backward(X, G, C5, out=out, workspace=ws)
    for i in range(3):
        X2, G2, _, _ = _batch("normal", 2, 200, 520, "bf16", 23 + i)
        X.copy_(X2)
        G.copy_(G2)
        want = mns.ns_orthogonalize_backward(X2, G2, C5)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), i


def test_two_streams_at_once():
    pairs = [_batch("normal", 1, 384, 640, "bf16", 29 + i)[:2] for i in range(2)]
    alone = [mns.ns_orthogonalize_backward(x, g, C5) for x, g in pairs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in pairs]
    got = [[mns.ns_orthogonalize_backward(x, g, C5, stream=s) for _ in range(3)]
           for (x, g), s in zip(pairs, streams)]
    torch.cuda.synchronize()
    for a, outs in zip(alone, got):
        for o in outs:
            assert torch.equal(o, a)


@pytest.mark.parametrize("dist", ["normal", "lowrank"])
@pytest.mark.parametrize("batch,rows,cols", [(1, 257, 300), (1, 300, 257), (3, 1111, 333),
                                             (2, 512, 512), (4, 512, 1030), (1, 400, 6000)])
def test_small_bfloat16_within_half_a_step(batch, rows, cols, dist):
    """The arithmetic's error together with the output's rounding stays below the largest rounding
    of a bfloat16 output alone (2^-8 of a value; its mean over a matrix is below half of that), for
    near-square and low-rank matrices too, where float16 shows most. Nothing is read from a
    workspace before it is written (filled with NaN), the padding among it."""
    _say("case", dist, batch, rows, cols)
    X, G, xs, gs = _batch(dist, batch, rows, cols, "bf16", 57)
    ws = torch.full((mns.ns_backward_workspace_size(X),), 0xFF, dtype=torch.uint8, device="cuda")
    dX = mns.ns_orthogonalize_backward(X, G, C5, workspace=ws)
    for i in range(batch):
        err = rel(to_f64(dX[i]), ref.gradient(xs[i], gs[i], C5))
        _say("  matrix", i, "error", f"{err:.2e}")
        assert err <= 2.0 ** -8


def test_last_chunk_of_another_form():
    """63 matrices: 32, then 31 in the form of small problems, on the workspace of the size asked
    for, against the same matrices in calls of their own chunk."""
    _say("case 63 x 300 x 570")
    g = torch.Generator().manual_seed(5)
    X = torch.randn(63, 300, 570, generator=g).bfloat16().cuda()
    G = torch.randn(63, 300, 570, generator=g).bfloat16().cuda()
    guard = 4096
    need = mns.ns_backward_workspace_size(X)
    room = torch.full((need + guard,), 0xFF, dtype=torch.uint8, device="cuda")
    dX = mns.ns_orthogonalize_backward(X, G, C5, workspace=room[:need])
    assert (room[need:] == 0xFF).all()
    assert torch.equal(dX[:32], mns.ns_orthogonalize_backward(X[:32], G[:32], C5))
    assert torch.equal(dX[32:], mns.ns_orthogonalize_backward(X[32:].clone(), G[32:].clone(), C5))
    for i in (0, 31, 32, 62):
        err = rel(to_f64(dX[i]), ref.gradient(X[i].double().cpu().numpy(), G[i].double().cpu().numpy(), C5))
        _say("  matrix", i, "error", f"{err:.2e}")
        assert err <= 2.0 ** -8


@pytest.mark.parametrize("coeffs", [[(70000.0, -1000.0, 0.0)], [(300.0, -500.0, 210.0), (1.5, -0.5, 0.0)],
                                    [(0.01, 0.0, 0.0), (100.0, 3.0, 0.0)], [(1e-3, 0.5, -0.25)] * 2],
                         ids=["large", "cancelling", "shrinking", "small"])
def test_coefficients_of_odd_sizes(coeffs):
    """Coefficients whose P passes float16's range, or whose iterations shrink a direction and let it
    grow again, in both forms of the float16 arithmetic and in float32."""
    for storage, batch, rows, cols in (("bf16", 1, 300, 500), ("bf16", 1, 900, 600), ("f32", 1, 130, 200)):
        X, G, xs, gs = _batch("normal", batch, rows, cols, storage, 71)
        if storage == "bf16" and coeffs[0][0] == 300.0:
            # f_1 reaches 94.1 and f_2 = 1.5 f_1 - 0.5 f_1^3 has the slope (1.5 - 1.5 f_1^2) f_1':
            # a direction grows 1.5e6 times, more than the 2^20 that float16 takes
            with pytest.raises(mns._abi.MnsError):
                mns.ns_orthogonalize_backward(X, G, coeffs)
            continue
        dX = mns.ns_orthogonalize_backward(X, G, coeffs)
        err = rel(to_f64(dX[0]), ref.gradient(xs[0], gs[0], coeffs))
        _say("case", storage, rows, cols, coeffs, f"error {err:.2e}")
        assert err <= TOL[storage]


RANGES = {
    "grown": [(70000.0, -1000.0, 0.0), (1.5, 0.0, 0.0)],
    "doubled": [(2.0, 0.0, 0.0)] * 10,
    "shrunk": [(0.01, 0.0, 0.0)] * 4,
    "down_and_up": [(1e-3, 0.0, 0.0), (1e-3, 0.0, 0.0), (900.0, -3e14, 0.0)],
    "up_and_down": [(300.0, 0.0, 0.0), (300.0, 0.0, 0.0), (1e-4, -5e-15, 0.0)],
    "float32": [(1e15, 0.0, 0.0), (1e14, 0.0, 0.0), (1e-10, 0.0, 0.0)],
}


@pytest.mark.parametrize("name", sorted(RANGES))
@pytest.mark.parametrize("kind", ["normal", "rank_one"])
def test_iterates_far_from_one(name, kind):
    """Iterations that take the singular values of X, and the directions, far above or below 1 and go on
    from there: what is stored in between (X, A = X X^T, E, P) stays in the range of its type, in every
    form of the arithmetic. In float16 one step of a value at the top of its range is 2^-11 of it."""
    coeffs = RANGES[name]
    for storage, rows, cols in (("bf16", 300, 500), ("bf16", 600, 900), ("bf16", 900, 600),
                                ("bf16", 40, 90), ("f32", 130, 200), ("f32", 600, 900), ("f32", 60, 200)):
        if name == "float32" and storage == "bf16":
            continue
        X, G, xs, gs = _batch("normal", 1, rows, cols, storage, 83)
        if kind == "rank_one":
            X[0] = (X[0, :, :1].float() @ X[0, :1].float()).to(X.dtype)
            xs = [to_f64(X[0])]
        dX = mns.ns_orthogonalize_backward(X, G, coeffs)
        err = rel(to_f64(dX[0]), ref.gradient(xs[0], gs[0], coeffs))
        _say("case", name, kind, storage, rows, cols, f"error {err:.2e}")
        assert err <= TOL[storage]


@pytest.mark.parametrize("dist", ["normal", "lowrank"])
@pytest.mark.parametrize("batch,rows,cols", [(1, 513, 513), (1, 700, 700), (1, 900, 600), (3, 600, 900),
                                             (1, 1024, 1024), (1, 1024, 4096), (12, 512, 1100)])
def test_larger_bfloat16_within_half_a_step(batch, rows, cols, dist):
    """As test_small_bfloat16_within_half_a_step, where the products run on float16 operands of one
    part each: arithmetic and output rounding together stay below 2^-8 of the gradient, the largest
    rounding of a bfloat16 value."""
    _say("case", dist, batch, rows, cols)
    X, G, xs, gs = _batch(dist, batch, rows, cols, "bf16", 91)
    ws = torch.full((mns.ns_backward_workspace_size(X),), 0xFF, dtype=torch.uint8, device="cuda")
    dX = mns.ns_orthogonalize_backward(X, G, C5, workspace=ws)
    for i in range(0, batch, max(1, batch // 3)):
        err = rel(to_f64(dX[i]), ref.gradient(xs[i], gs[i], C5))
        _say("  matrix", i, "error", f"{err:.2e}")
        assert err <= 2.0 ** -8


@pytest.mark.parametrize("coeffs", [[(1e-38, 0.0, 0.0)] * 3, [(0.0, 0.0, 0.0)] * 2,
                                    [(0.0, 0.0, 0.0), (3.0, -1.0, 0.0)], [(1e-44, 0.0, 0.0)] * 4],
                         ids=["tiny", "zero", "zero_first", "denormal"])
def test_coefficients_that_leave_nothing(coeffs):
    """The gradient is zero, or below anything its type can hold: zeros, not NaN."""
    for storage, rows, cols in (("bf16", 300, 500), ("bf16", 600, 900), ("bf16", 40, 90),
                                ("f32", 130, 200), ("f32", 600, 900), ("f32", 60, 200)):
        X, G, _, _ = _batch("normal", 1, rows, cols, storage, 83)
        _say("case", storage, rows, cols, coeffs)
        assert not mns.ns_orthogonalize_backward(X, G, coeffs).any()
