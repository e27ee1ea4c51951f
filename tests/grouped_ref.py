"""Plain float64 forms of the products grouped by expert, with the error an implementation may
make: results and bounds element by element.

Bound of one element sum_i x_i y_i of r terms, added in float32 in any order: every product and
every addition is off by at most one unit in the last place of float32 (2^-23 relative; half a
unit when rounded to nearest, a whole one whichever way the matrix unit rounds), so the sum is
off by at most (r + 2) 2^-23 sum |x_i y_i|. Storing it in bfloat16 adds half a step, 2^-8 of
the value; beta C adds one product and one addition."""
import torch

ULP = 2.0 ** -23
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def bounds_of(sizes, front=0):
    b = [front]
    for s in sizes:
        b.append(b[-1] + s)
    return b


def stored(v, err, dtype):
    """Error bound of v (off by err) once rounded to dtype."""
    return err + HALF_STEP[dtype] * (v.abs() + err) + 1e-38


def matmul(X, W, bounds, transpose_w, start):
    """(result, bound): rows of no expert keep `start`."""
    Xd, Wd = X.cpu().double(), W.cpu().double()
    out = start.cpu().double().clone()
    err = torch.zeros_like(out)
    r = Xd.shape[1]
    for e, (lo, hi) in enumerate(zip(bounds, bounds[1:])):
        w = Wd[e] if transpose_w else Wd[e].t()
        out[lo:hi] = Xd[lo:hi] @ w
        err[lo:hi] = stored(out[lo:hi], (r + 2) * ULP * (Xd[lo:hi].abs() @ w.abs()), X.dtype)
    return out, err


def weight_grad(dY, X, bounds, C, beta, dtype):
    dYd, Xd = dY.cpu().double(), X.cpu().double()
    e = len(bounds) - 1
    out = torch.zeros(e, dY.shape[1], X.shape[1], dtype=torch.float64)
    err = torch.zeros_like(out)
    for i, (lo, hi) in enumerate(zip(bounds, bounds[1:])):
        out[i] = dYd[lo:hi].t() @ Xd[lo:hi]
        mag = dYd[lo:hi].abs().t() @ Xd[lo:hi].abs()
        if C is not None and beta != 0.0:
            out[i] += beta * C[i].cpu().double()
            mag += abs(beta) * C[i].cpu().double().abs()
        err[i] = stored(out[i], (hi - lo + 3) * ULP * mag, dtype)
    return out, err


def check(got, ref, err, what=""):
    got = got.cpu().double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    over = ((got - ref).abs() - err).max().item() if got.numel() else 0.0
    assert over <= 0.0, f"{what}: {over:.3g} beyond the bound"
