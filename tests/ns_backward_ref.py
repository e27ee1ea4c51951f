"""Gradient of O = NS_T(X / ||X||_F) in float64, two ways: walking back through the stored
iterates, and the closed form in the singular basis."""
import numpy as np


def forward(X, coeffs):
    X = np.asarray(X, dtype=np.float64)
    n = np.linalg.norm(X)
    Y = X / n if n > 0 else np.zeros_like(X)
    if tall := Y.shape[0] > Y.shape[1]:
        Y = Y.T
    for a, b, c in coeffs:
        A = Y @ Y.T
        Y = a * Y + (b * A + c * (A @ A)) @ Y
    return Y.T if tall else Y


def gradient(X, G, coeffs):
    """Reverse mode: X' = P X with P = a I + b A + c A^2 gives dX = P G + (N + N^T) X for
    N = b K + c (A K + K A), K = G X^T."""
    X, G = np.asarray(X, dtype=np.float64), np.asarray(G, dtype=np.float64)
    norm = np.linalg.norm(X)
    if norm == 0.0:
        return np.zeros_like(X)
    if tall := X.shape[0] > X.shape[1]:
        X, G = X.T, G.T
    X0 = X / norm
    kept, Y = [], X0
    for a, b, c in coeffs:
        A = Y @ Y.T
        P = a * np.eye(len(A)) + b * A + c * (A @ A)
        kept.append((Y, A, P))
        Y = P @ Y
    for (a, b, c), (Y, A, P) in zip(reversed(list(coeffs)), reversed(kept)):
        K = G @ Y.T
        N = b * K + c * (A @ K + K @ A)
        G = P @ G + (N + N.T) @ Y
    out = (G - X0 * np.sum(X0 * G)) / norm
    return out.T if tall else out


def gradient_svd(X, G, coeffs):
    """Closed form for a matrix with distinct positive singular values."""
    X, G = np.asarray(X, dtype=np.float64), np.asarray(G, dtype=np.float64)
    if tall := X.shape[0] > X.shape[1]:
        X, G = X.T, G.T
    norm = np.linalg.norm(X)
    U, s, Vt = np.linalg.svd(X / norm, full_matrices=True)
    n = len(s)
    f, d = s.copy(), np.ones_like(s)
    for a, b, c in coeffs:
        d *= a + 3 * b * f ** 2 + 5 * c * f ** 4
        f = a * f + b * f ** 3 + c * f ** 5
    E = U.T @ G @ Vt.T
    sq, rest = E[:, :n], E[:, n:]
    si, sj, fi, fj = s[:, None], s[None, :], f[:, None], f[None, :]
    eye = np.eye(n, dtype=bool)
    diff = np.where(eye, d[:, None], (fi - fj) / np.where(eye, 1.0, si - sj))
    out = diff * (sq + sq.T) / 2 + (fi + fj) / (si + sj) * (sq - sq.T) / 2
    J = U @ np.hstack([out, (f / s)[:, None] * rest]) @ Vt
    X0 = X / norm
    J = (J - X0 * np.sum(X0 * J)) / norm
    return J.T if tall else J
