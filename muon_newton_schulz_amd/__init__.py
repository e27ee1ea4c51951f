"""MI355X (gfx950) Muon / Newton-Schulz / Gram-NS / NorMuon / Dion3 optimizer step.

Thin Python binding over the C ABI in include/muon_ns.h: it turns torch tensors into
device pointers and sizes and calls the HIP library; every step of the computation runs in
the library's kernels. PyTorch supplies device memory and the current stream only. The
library must be built (``python -m muon_newton_schulz_amd.build``); there is no fallback.
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import Iterable, Sequence

import torch

from . import _abi
from ._abi import (MNS_BF16, MNS_F32, MNS_NS_GRAM, MNS_NS_STANDARD, MnsError,  # noqa: F401
                   MnsHparams, MnsMatrix, check, load)

__all__ = ["muon_step", "ns_orthogonalize", "ns_orthogonalize_noalloc",
           "gram_ns_orthogonalize", "normuon_scale",
           "ns_orthogonalize_backward", "ns_backward_workspace_size",
           "grouped_matmul", "grouped_weight_grad", "muon_step_grouped",
           "grouped_step_workspace_size",
           "step_workspace_size", "ns_workspace_size", "normuon_workspace_size",
           "restart_mask", "profile_begin", "profile_set_flush", "profile_end", "MnsError",
           "load"]

_KINDS = {"standard": MNS_NS_STANDARD, "gram": MNS_NS_GRAM}


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return MNS_BF16
    if t.dtype == torch.float32:
        return MNS_F32
    raise TypeError(f"unsupported storage dtype {t.dtype} (bfloat16 or float32)")


def _ptr(t: torch.Tensor | None) -> int | None:
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


def _on_one_gpu(tensors, what: str) -> torch.device:
    """Every tensor must live on one CUDA (HIP) device: a host pointer handed to a kernel
    faults the GPU. Returns that device."""
    dev = None
    for t in tensors:
        if t is None:
            continue
        if t.device.type != "cuda":
            raise ValueError(f"{what}: every tensor must be on a GPU (got {t.device})")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError(f"{what}: tensors on different devices ({dev} and {t.device})")
    return dev


def _span(t: torch.Tensor):
    n = t.numel() * t.element_size()
    return t.data_ptr(), t.data_ptr() + n


def _disjoint(a: torch.Tensor, b: torch.Tensor) -> bool:
    a0, a1 = _span(a)
    b0, b1 = _span(b)
    return a1 <= b0 or b1 <= a0


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _coeffs(coeffs: Sequence[Sequence[float]]):
    flat = [float(c) for abc in coeffs for c in abc]
    if len(flat) != 3 * len(coeffs):
        raise ValueError("each iteration needs (a_t, b_t, c_t)")
    return (ctypes.c_float * max(1, len(flat)))(*flat), len(coeffs)


# The restart mask is a 32-bit field: restarts can be placed before iterations 2 .. 31.
MAX_RESTART_ITERATION = 31


def restart_mask(restart_before: Iterable[int], T: int | None = None) -> int:
    """Bit t set = restart before iteration t (Gram Newton-Schulz). Raises for an iteration
    outside 2 .. min(T, 31) (T given) or 2 .. 31."""
    hi = MAX_RESTART_ITERATION if T is None else min(int(T), MAX_RESTART_ITERATION)
    mask = 0
    for t in restart_before:
        t = int(t)
        if not 2 <= t <= hi:
            raise ValueError(f"restart before iteration {t}: must lie in 2..{hi}")
        mask |= 1 << t
    return mask


def _workspace(nbytes: int, device, workspace: torch.Tensor | None) -> torch.Tensor:
    if workspace is not None:
        if workspace.device != device:
            raise ValueError(f"workspace on {workspace.device}, tensors on {device}")
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
        if workspace.numel() * workspace.element_size() < nbytes:
            raise ValueError(f"workspace too small: need {nbytes} bytes")
        return workspace
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


def _as_list(x):
    if x is None:
        return None
    return list(x) if isinstance(x, (list, tuple)) else [x]


def _hparams(dtype: int, mu, lr, coeffs, kind, restart_before, normuon, beta2, eps,
             row_fraction):
    abc, T = _coeffs(coeffs)
    if kind not in _KINDS:
        raise ValueError(f"kind must be one of {sorted(_KINDS)}")
    hp = MnsHparams(mu=mu, lr=lr, T=T, abc=ctypes.cast(abc, ctypes.POINTER(ctypes.c_float)),
                    kind=_KINDS[kind], restart_mask=restart_mask(restart_before, T),
                    normuon=1 if normuon else 0, beta2=beta2, eps=eps,
                    row_fraction=row_fraction, dtype=dtype)
    return hp, abc


def _first_dtype(W) -> int:
    Ws = _as_list(W)
    if not Ws:
        raise ValueError("no matrices")
    return _dtype_code(Ws[0])


def _matrices(W, M, G, v, normuon: bool):
    """Checks the step's tensors and packs them into the ABI's matrix array. The library
    applies one storage dtype to every W and G of a call and reads v as float32 [rows], so
    a mismatch here would make its kernels read or write out of bounds."""
    Ws, Ms, Gs, vs = _as_list(W), _as_list(M), _as_list(G), _as_list(v)
    if not Ws:
        raise ValueError("no matrices")
    if not (len(Ws) == len(Ms) == len(Gs)) or (vs is not None and len(vs) != len(Ws)):
        raise ValueError("W, M, G (and v) must have the same number of matrices")
    if normuon and vs is None:
        raise ValueError("NorMuon needs v (one float32 vector per matrix)")
    dtype = Ws[0].dtype
    _dtype_code(Ws[0])
    for i, (w, m, g) in enumerate(zip(Ws, Ms, Gs)):
        if w.dim() != 2 or w.shape != m.shape or w.shape != g.shape:
            raise ValueError(f"matrix {i}: W, M and G must be 2-D tensors of the same shape")
        if w.dtype != dtype or g.dtype != dtype:
            raise TypeError(f"matrix {i}: W and G must all share one storage dtype ({dtype}); "
                            f"got W {w.dtype}, G {g.dtype}")
        if m.dtype != torch.float32:
            raise TypeError(f"matrix {i}: momentum must be float32")
        if vs is not None:
            vi = vs[i]
            if vi.dtype != torch.float32 or vi.dim() != 1 or vi.shape[0] != w.shape[0]:
                raise ValueError(f"matrix {i}: v must be float32 of shape ({w.shape[0]},)")
        for t in (w, m, g) + ((vs[i],) if vs is not None else ()):
            if not t.is_contiguous():
                raise ValueError(f"matrix {i}: tensors must be contiguous")
    dev = _on_one_gpu(Ws + Ms + Gs + (vs or []), "muon_step")
    arr = (MnsMatrix * len(Ws))()
    for i, (w, m, g) in enumerate(zip(Ws, Ms, Gs)):
        arr[i].W = _ptr(w)
        arr[i].M = _ptr(m)
        arr[i].G = _ptr(g)
        arr[i].v = _ptr(vs[i]) if vs is not None else None
        arr[i].rows, arr[i].cols = w.shape
    return arr, Ws, dev


def step_workspace_size(W, M, G, v=None, *, mu=0.95, lr=0.02, coeffs, kind="standard",
                        restart_before=(), normuon=False, beta2=0.95, eps=1e-8,
                        row_fraction=1.0) -> int:
    hp, _keep = _hparams(_first_dtype(W), mu, lr, coeffs, kind, restart_before, normuon,
                         beta2, eps, row_fraction)
    arr, Ws, _dev = _matrices(W, M, G, v, normuon)
    out = ctypes.c_size_t(0)
    check(load().mns_step_workspace_size(arr, len(Ws), ctypes.byref(hp), ctypes.byref(out)),
          "mns_step_workspace_size")
    return out.value


def muon_step(W, M, G, v=None, *, mu: float, lr: float, coeffs, kind: str = "standard",
              restart_before=(), normuon: bool = False, beta2: float = 0.95,
              eps: float = 1e-8, row_fraction: float = 1.0,
              workspace: torch.Tensor | None = None, stream=None) -> None:
    """One optimizer step, in place on W, M (and v), over one matrix or a list of them.

    Eq. (1) of the Dion3 page; NorMuon (Eq. 2) when ``normuon``; Dion3 fractional row
    selection (Algorithm 4) when ``row_fraction`` < 1 (``lr`` is used as given)."""
    hp, _keep = _hparams(_first_dtype(W), mu, lr, coeffs, kind, restart_before, normuon,
                         beta2, eps, row_fraction)
    arr, Ws, dev = _matrices(W, M, G, v, normuon)
    lib = load()
    need = ctypes.c_size_t(0)
    check(lib.mns_step_workspace_size(arr, len(Ws), ctypes.byref(hp), ctypes.byref(need)),
          "mns_step_workspace_size")
    ws = _workspace(need.value, dev, workspace)
    check(lib.muon_step(arr, len(Ws), ctypes.byref(hp), ws.data_ptr(),
                        ws.numel() * ws.element_size(), _stream(stream)), "muon_step")


def ns_workspace_size(X: torch.Tensor, kind: str = "standard") -> int:
    b, r, c = _bshape(X)
    out = ctypes.c_size_t(0)
    check(load().mns_ns_workspace_size(_dtype_code(X), b, r, c, _KINDS[kind],
                                       ctypes.byref(out)), "mns_ns_workspace_size")
    return out.value


def _bshape(X: torch.Tensor):
    if X.dim() == 2:
        return 1, X.shape[0], X.shape[1]
    if X.dim() == 3:
        return X.shape[0], X.shape[1], X.shape[2]
    raise ValueError("X must be 2-D or a 3-D batch")


def _ns_operands(X: torch.Tensor, out: torch.Tensor | None, what: str):
    """X (2-D, or a 3-D batch) in a storage dtype on one GPU, and the output: a new tensor
    like X, or `out`, which must match X in shape, dtype and device and not overlap it."""
    b, r, c = _bshape(X)
    _dtype_code(X)
    if not X.is_contiguous():
        raise ValueError(f"{what}: X must be contiguous")
    if out is not None:
        if out.shape != X.shape or out.dtype != X.dtype:
            raise ValueError(f"{what}: out must match X in shape and dtype "
                             f"(X {tuple(X.shape)} {X.dtype}, out {tuple(out.shape)} {out.dtype})")
        if not out.is_contiguous():
            raise ValueError(f"{what}: out must be contiguous")
    if out is not None and not _disjoint(X, out):
        raise ValueError(f"{what}: out may not overlap X")
    _on_one_gpu([X, out], what)
    O = torch.empty_like(X) if out is None else out
    return b, r, c, O


def ns_orthogonalize(X: torch.Tensor, coeffs, out: torch.Tensor | None = None,
                     workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Standard quintic Newton-Schulz of X / ||X||_F (per matrix of a batch)."""
    b, r, c, O = _ns_operands(X, out, "ns_orthogonalize")
    abc, T = _coeffs(coeffs)
    lib = load()
    ws = _workspace(ns_workspace_size(X, "standard"), X.device, workspace)
    check(lib.ns_orthogonalize(_ptr(X), _ptr(O), _dtype_code(X), b, r, c, T, abc,
                               ws.data_ptr(), ws.numel() * ws.element_size(), _stream(stream)),
          "ns_orthogonalize")
    return O


def ns_orthogonalize_noalloc(X: torch.Tensor, coeffs, out: torch.Tensor, stream=None) -> torch.Tensor:
    """ns_orthogonalize without a workspace: the library's own device scratch (64 MiB per GPU)
    holds every buffer, so the call allocates nothing (graph capture, serving loops). `out`
    must be given; overlapping calls on one GPU race."""
    if out is None:
        raise ValueError("ns_orthogonalize_noalloc: out must be given (nothing is allocated)")
    b, r, c, O = _ns_operands(X, out, "ns_orthogonalize_noalloc")
    abc, T = _coeffs(coeffs)
    check(load().ns_orthogonalize_noalloc(_ptr(X), _ptr(O), _dtype_code(X), b, r, c, T, abc,
                                          _stream(stream)), "ns_orthogonalize_noalloc")
    return O


def gram_ns_orthogonalize(X: torch.Tensor, coeffs, restart_before=(3,),
                          out: torch.Tensor | None = None,
                          workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Gram Newton-Schulz (Theorem 2 with restarts) of X / ||X||_F."""
    b, r, c, O = _ns_operands(X, out, "gram_ns_orthogonalize")
    abc, T = _coeffs(coeffs)
    mask = restart_mask(restart_before, T)
    lib = load()
    ws = _workspace(ns_workspace_size(X, "gram"), X.device, workspace)
    check(lib.gram_ns_orthogonalize(_ptr(X), _ptr(O), _dtype_code(X), b, r, c, T, abc,
                                    mask, ws.data_ptr(),
                                    ws.numel() * ws.element_size(), _stream(stream)),
          "gram_ns_orthogonalize")
    return O


def normuon_workspace_size(O: torch.Tensor) -> int:
    b, r, c = _bshape(O)
    out = ctypes.c_size_t(0)
    check(load().mns_normuon_workspace_size(b, r, c, ctypes.byref(out)),
          "mns_normuon_workspace_size")
    return out.value


def normuon_scale(O: torch.Tensor, v: torch.Tensor, beta2: float = 0.95, eps: float = 1e-8,
                  workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """NorMuon normalisation (Eq. 2) of O in place; v (float32, one per row) is updated."""
    b, r, c = _bshape(O)
    _dtype_code(O)
    if v.dtype != torch.float32 or v.numel() != b * r:
        raise ValueError("v must be float32 with one entry per row")
    if not O.is_contiguous() or not v.is_contiguous():
        raise ValueError("normuon_scale: O and v must be contiguous")
    if not _disjoint(O, v):
        raise ValueError("normuon_scale: v may not overlap O")
    _on_one_gpu([O, v], "normuon_scale")
    lib = load()
    ws = _workspace(normuon_workspace_size(O), O.device, workspace)
    check(lib.normuon_scale(_ptr(O), _dtype_code(O), b, r, c,
                            ctypes.cast(_ptr(v), ctypes.POINTER(ctypes.c_float)), beta2, eps,
                            ws.data_ptr(), ws.numel() * ws.element_size(), _stream(stream)),
          "normuon_scale")
    return O


class _OnStream:
    """The device of a call's tensors and the stream it runs on (a torch stream, a raw
    hipStream_t, or None for that device's current stream). Inside the context the device is
    current and torch allocates on that stream, so an output or workspace made there is not
    handed out again before the call's kernels are done with it."""

    def __init__(self, device: torch.device, stream):
        self._ctx = None
        if stream is None:
            if device.index != torch.cuda.current_device():
                self._ctx = torch.cuda.device(device)
            # the current stream's handle, without building a stream object around it (3.5 us of a
            # small call's 12)
            self.handle = torch._C._cuda_getCurrentRawStream(device.index)
            return
        if not hasattr(stream, "cuda_stream"):
            handle = int(stream)
            if handle == 0:
                stream = torch.cuda.default_stream(device)
            else:
                stream = torch.cuda.ExternalStream(handle, device=device)
        elif stream.device != device:
            raise ValueError(f"stream on {stream.device}, tensors on {device}")
        self.handle = stream.cuda_stream
        self._ctx = contextlib.ExitStack()
        self._ctx.enter_context(torch.cuda.device(device))
        self._ctx.enter_context(torch.cuda.stream(stream))

    def __enter__(self):
        if isinstance(self._ctx, torch.cuda.device):
            self._ctx.__enter__()
        return self.handle

    def __exit__(self, *exc):
        if self._ctx is not None:
            self._ctx.__exit__(*exc)
        return False


def _pitch(t: torch.Tensor, name: str, what: str) -> int:
    """Row pitch of a 2-D tensor whose rows are contiguous and do not overlap."""
    rows, cols = t.shape
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{what}: the rows of {name} must be contiguous")
    if rows <= 1:
        return cols
    if t.stride(0) < cols:
        raise ValueError(f"{what}: the rows of {name} overlap")
    return t.stride(0)


def _extent(t: torch.Tensor):
    """First byte and the byte behind the last one a (strided) tensor reaches."""
    if t.numel() == 0:
        return 0, 0
    last = sum((n - 1) * s for n, s in zip(t.shape, t.stride()))
    return t.data_ptr(), t.data_ptr() + (last + 1) * t.element_size()


def _apart(a: torch.Tensor, b: torch.Tensor) -> bool:
    a0, a1 = _extent(a)
    b0, b1 = _extent(b)
    return a1 <= b0 or b1 <= a0


def _grouped_checks(tokens, stack, offsets, groups: int, what: str) -> torch.device:
    for name, t in tokens:
        if t.dim() != 2:
            raise ValueError(f"{what}: {name} must be 2-D (rows x width)")
    if offsets.dim() != 1 or offsets.dtype != torch.int64 or offsets.shape[0] != groups + 1:
        raise ValueError(f"{what}: offsets must be int64 of shape ({groups + 1},)")
    if not offsets.is_contiguous():
        raise ValueError(f"{what}: offsets must be contiguous")
    return _on_one_gpu([t for _, t in tokens] + list(stack) + [offsets], what)


def _grouped_workspace(weight_grad: int, code: int, groups: int, rows: int, n: int, k: int,
                       device, workspace):
    need = ctypes.c_size_t(0)
    check(load().mns_grouped_workspace_size(weight_grad, code, groups, rows, n, k,
                                            ctypes.byref(need)), "mns_grouped_workspace_size")
    if need.value == 0:
        return None, 0, 0
    ws = _workspace(need.value, device, workspace)
    return ws, ws.data_ptr(), ws.numel() * ws.element_size()


def grouped_matmul(X: torch.Tensor, W: torch.Tensor, offsets: torch.Tensor, *,
                   transpose_w: bool = False, out: torch.Tensor | None = None,
                   workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Rows sorted by expert times their expert's matrix: Y_e = X_e W_e^T (the forward product
    of a layer of experts), or Y_e = X_e W_e with ``transpose_w`` (the gradient of its input).

    W is a contiguous (experts, n, k) stack; expert e owns rows offsets[e]:offsets[e + 1] of X
    (offsets: int64 on the GPU, read by the kernels only). X and ``out`` are 2-D with contiguous
    rows at any row pitch. Rows that belong to no expert come back as zeros in a new output and
    are left as they are in a given ``out``.

    Autograd does not see the call (its result never requires grad): the gradients are calls of
    their own, ``transpose_w`` for X's and grouped_weight_grad for W's."""
    what = "grouped_matmul"
    if W.dim() != 3:
        raise ValueError(f"{what}: W must be 3-D (experts, n, k)")
    code = _dtype_code(X)
    if W.dtype != X.dtype:
        raise TypeError(f"{what}: X and W must share one storage dtype "
                        f"(X {X.dtype}, W {W.dtype})")
    groups, n, k = W.shape
    wide, narrow = (n, k) if transpose_w else (k, n)
    if X.dim() != 2 or X.shape[1] != wide:
        raise ValueError(f"{what}: X must be 2-D with rows of {wide}, got {tuple(X.shape)}")
    if not W.is_contiguous():
        raise ValueError(f"{what}: W must be contiguous")
    rows = X.shape[0]
    ldx = _pitch(X, "X", what)
    if out is not None:
        if out.dim() != 2 or tuple(out.shape) != (rows, narrow) or out.dtype != X.dtype:
            raise ValueError(f"{what}: out must be {(rows, narrow)} {X.dtype}, "
                             f"got {tuple(out.shape)} {out.dtype}")
        ldy = _pitch(out, "out", what)
        if not _apart(out, X) or not _apart(out, W) or not _apart(out, offsets):
            raise ValueError(f"{what}: out may not overlap X, W or offsets")
    dev = _grouped_checks([("X", X)] + ([("out", out)] if out is not None else []), [W], offsets,
                          groups, what)
    with _OnStream(dev, stream) as handle:
        Y = out
        if Y is None:
            Y = torch.empty((rows, narrow), dtype=X.dtype, device=dev)
            ldy = narrow
        keep, ws, nbytes = _grouped_workspace(0, code, groups, rows, n, k, dev, workspace)
        check(load().grouped_matmul(X.data_ptr(), ldx, W.data_ptr(), Y.data_ptr(), ldy, code,
                                    offsets.data_ptr(), groups, rows, n, k,
                                    1 if transpose_w else 0, 1 if out is None else 0, ws, nbytes,
                                    handle), what)
    return Y


def grouped_weight_grad(dY: torch.Tensor, X: torch.Tensor, offsets: torch.Tensor, *,
                        C: torch.Tensor | None = None, beta: float = 1.0,
                        out: torch.Tensor | None = None, out_dtype: torch.dtype | None = None,
                        workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Weight gradients of a layer of experts, G_e = beta C_e + dY_e^T X_e, as a stack
    (experts, n, k) for dY of width n and X of width k, rows sorted by expert as in
    grouped_matmul. The output is of ``out``'s dtype, else C's, else ``out_dtype``, else X's;
    float32 outputs take bfloat16 products unrounded. ``out`` may be C itself: with a float32
    momentum, ``C=M, beta=mu, out=M`` is M <- mu M + dY^T X. Autograd does not see the call."""
    what = "grouped_weight_grad"
    code = _dtype_code(X)
    if dY.dtype != X.dtype:
        raise TypeError(f"{what}: dY and X must share one storage dtype "
                        f"(dY {dY.dtype}, X {X.dtype})")
    if dY.dim() != 2 or X.dim() != 2 or dY.shape[0] != X.shape[0]:
        raise ValueError(f"{what}: dY and X must be 2-D with the same rows")
    if offsets.dim() != 1 or offsets.shape[0] < 2:
        raise ValueError(f"{what}: offsets must hold at least two entries")
    rows, n, k, groups = X.shape[0], dY.shape[1], X.shape[1], offsets.shape[0] - 1
    lddy, ldx = _pitch(dY, "dY", what), _pitch(X, "X", what)
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else C.dtype if C is not None else X.dtype
    for name, t in (("C", C), ("out", out)):
        if t is None:
            continue
        if tuple(t.shape) != (groups, n, k) or t.dtype != out_dtype:
            raise ValueError(f"{what}: {name} must be {(groups, n, k)} {out_dtype}, "
                             f"got {tuple(t.shape)} {t.dtype}")
        if not t.is_contiguous():
            raise ValueError(f"{what}: {name} must be contiguous")
    if out_dtype not in (X.dtype, torch.float32):
        raise TypeError(f"{what}: the output must be {X.dtype} or float32, not {out_dtype}")
    if out is not None:
        if not _apart(out, dY) or not _apart(out, X) or not _apart(out, offsets):
            raise ValueError(f"{what}: out may not overlap dY, X or offsets")
        if C is not None and C.data_ptr() != out.data_ptr() and not _apart(out, C):
            raise ValueError(f"{what}: out must be C itself or lie apart from it")
    dev = _grouped_checks([("dY", dY), ("X", X)], [t for t in (C, out) if t is not None], offsets,
                          groups, what)
    with _OnStream(dev, stream) as handle:
        G = torch.empty((groups, n, k), dtype=out_dtype, device=dev) if out is None else out
        keep, ws, nbytes = _grouped_workspace(1, code, groups, rows, n, k, dev, workspace)
        check(load().grouped_weight_grad(dY.data_ptr(), lddy, X.data_ptr(), ldx, code,
                                         offsets.data_ptr(), groups, rows, n, k,
                                         None if C is None else C.data_ptr(), beta, G.data_ptr(),
                                         MNS_F32 if out_dtype == torch.float32 else MNS_BF16, ws,
                                         nbytes, handle), what)
    return G


def _grouped_step(W, M, dY, X, offsets, v, normuon, what):
    """Checks of muon_step_grouped's tensors: device, sizes and row pitches."""
    if W.dim() != 3 or W.shape != M.shape:
        raise ValueError(f"{what}: W and M must be 3-D stacks (experts, rows, cols) of one shape")
    _dtype_code(W)
    if M.dtype != torch.float32:
        raise TypeError(f"{what}: momentum must be float32")
    if dY.dtype != W.dtype or X.dtype != W.dtype:
        raise TypeError(f"{what}: W, dY and X must share one storage dtype (W {W.dtype}, "
                        f"dY {dY.dtype}, X {X.dtype})")
    groups, rows, cols = W.shape
    if dY.dim() != 2 or X.dim() != 2 or dY.shape[0] != X.shape[0]:
        raise ValueError(f"{what}: dY and X must be 2-D with the same rows")
    if dY.shape[1] != rows or X.shape[1] != cols:
        raise ValueError(f"{what}: dY must have rows of {rows} and X of {cols}")
    if normuon and v is None:
        raise ValueError("NorMuon needs v (float32, one entry per expert and row)")
    if v is not None and (v.dtype != torch.float32 or tuple(v.shape) != (groups, rows)):
        raise ValueError(f"{what}: v must be float32 of shape ({groups}, {rows})")
    state = [t for t in (W, M, v) if t is not None]
    if not all(t.is_contiguous() for t in state):
        raise ValueError(f"{what}: W, M and v must be contiguous")
    lddy, ldx = _pitch(dY, "dY", what), _pitch(X, "X", what)
    for i, a in enumerate(state):
        for b in state[i + 1:] + [dY, X, offsets]:
            if not _apart(a, b):
                raise ValueError(f"{what}: W, M and v may not overlap each other or the inputs")
    dev = _grouped_checks([("dY", dY), ("X", X)], state, offsets, groups, what)
    return dev, groups, X.shape[0], rows, cols, lddy, ldx


def grouped_step_workspace_size(W, M, dY, X, offsets, v=None, *, mu=0.95, lr=0.02, coeffs,
                                kind="standard", restart_before=(), normuon=False, beta2=0.95,
                                eps=1e-8) -> int:
    what = "grouped_step_workspace_size"
    hp, _keep = _hparams(_dtype_code(W), mu, lr, coeffs, kind, restart_before, normuon, beta2, eps,
                         1.0)
    _dev, groups, total, rows, cols, _a, _b = _grouped_step(W, M, dY, X, offsets, v, normuon, what)
    out = ctypes.c_size_t(0)
    check(load().mns_grouped_step_workspace_size(groups, total, rows, cols, ctypes.byref(hp),
                                                 ctypes.byref(out)),
          "mns_grouped_step_workspace_size")
    return out.value


def muon_step_grouped(W, M, dY, X, offsets, v=None, *, mu: float, lr: float, coeffs,
                      kind: str = "standard", restart_before=(), normuon: bool = False,
                      beta2: float = 0.95, eps: float = 1e-8,
                      workspace: torch.Tensor | None = None, stream=None) -> None:
    """One optimizer step, in place on W, M (and v), for a stack of experts (experts, rows, cols)
    whose gradients dY_e^T X_e are given by their tokens, sorted by expert as in grouped_matmul,
    and are never formed: the product adds them to the float32 momentum. M is a float32 stack like
    W, v float32 (experts, rows). Otherwise as muon_step (no row selection)."""
    what = "muon_step_grouped"
    hp, _keep = _hparams(_dtype_code(W), mu, lr, coeffs, kind, restart_before, normuon, beta2, eps,
                         1.0)
    dev, groups, total, rows, cols, lddy, ldx = _grouped_step(W, M, dY, X, offsets, v, normuon,
                                                              what)
    lib = load()
    need = ctypes.c_size_t(0)
    check(lib.mns_grouped_step_workspace_size(groups, total, rows, cols, ctypes.byref(hp),
                                              ctypes.byref(need)),
          "mns_grouped_step_workspace_size")
    with _OnStream(dev, stream) as handle:
        ws = _workspace(need.value, dev, workspace)
        check(lib.muon_step_grouped(W.data_ptr(), M.data_ptr(), None if v is None else v.data_ptr(),
                                    dY.data_ptr(), lddy, X.data_ptr(), ldx, offsets.data_ptr(),
                                    groups, total, rows, cols, ctypes.byref(hp), ws.data_ptr(),
                                    ws.numel() * ws.element_size(), handle), what)


def ns_backward_workspace_size(X: torch.Tensor) -> int:
    b, r, c = _bshape(X)
    out = ctypes.c_size_t(0)
    check(load().mns_ns_backward_workspace_size(_dtype_code(X), b, r, c, ctypes.byref(out)),
          "mns_ns_backward_workspace_size")
    return out.value


def ns_orthogonalize_backward(X: torch.Tensor, dO: torch.Tensor, coeffs,
                              out: torch.Tensor | None = None,
                              workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Gradient dX of ns_orthogonalize(X, coeffs) for the gradient dO of its output (the same for
    gram_ns_orthogonalize, whose map is the same). X and dO: one matrix or a 3-D batch, of one
    shape and storage dtype; X is the forward call's input, nothing else is kept from it. Autograd
    sees neither the forward call nor this one."""
    what = "ns_orthogonalize_backward"
    if dO.shape != X.shape or dO.dtype != X.dtype:
        raise ValueError(f"{what}: dO must match X in shape and dtype "
                         f"(X {tuple(X.shape)} {X.dtype}, dO {tuple(dO.shape)} {dO.dtype})")
    if not dO.is_contiguous():
        raise ValueError(f"{what}: dO must be contiguous")
    b, r, c = _bshape(X)
    code = _dtype_code(X)
    if not X.is_contiguous():
        raise ValueError(f"{what}: X must be contiguous")
    if out is not None:
        if out.shape != X.shape or out.dtype != X.dtype or not out.is_contiguous():
            raise ValueError(f"{what}: out must match X in shape and dtype and be contiguous")
        if not _disjoint(X, out) or not _disjoint(dO, out):
            raise ValueError(f"{what}: out may not overlap X or dO")
    dev = _on_one_gpu([X, dO, out], what)
    abc, T = _coeffs(coeffs)
    with _OnStream(dev, stream) as handle:
        dX = torch.empty_like(X) if out is None else out
        ws = _workspace(ns_backward_workspace_size(X), dev, workspace)
        check(load().ns_orthogonalize_backward(_ptr(X), _ptr(dO), _ptr(dX), code, b, r, c, T, abc,
                                               ws.data_ptr(), ws.numel() * ws.element_size(),
                                               handle), what)
    return dX


def profile_begin() -> None:
    """Start bracketing every library kernel launch with hipEvents (see mns_profile_begin)."""
    check(load().mns_profile_begin(), "mns_profile_begin")


def profile_set_flush(buffer: torch.Tensor | None) -> None:
    """Flush caches before each HBM-bound launch of the open session by writing over
    `buffer` (a device tensor, >= 1 GiB to evict the Infinity Cache); None turns it off."""
    if buffer is None:
        check(load().mns_profile_set_flush(None, 0), "mns_profile_set_flush")
        return
    if buffer.device.type != "cuda" or not buffer.is_contiguous():
        raise ValueError("the flush buffer must be a contiguous GPU tensor")
    check(load().mns_profile_set_flush(buffer.data_ptr(), buffer.numel() * buffer.element_size()),
          "mns_profile_set_flush")


def profile_end() -> list[dict]:
    """Close the session; per kernel: launches, event ms, algorithmic FLOPs and bytes."""
    lib = load()
    cap = 64
    arr = (_abi.MnsKernelStat * cap)()
    n = ctypes.c_int(0)
    check(lib.mns_profile_end(arr, cap, ctypes.byref(n)), "mns_profile_end")
    return [{"name": arr[i].name.decode(), "launches": arr[i].launches, "ms": arr[i].ms,
             "flops": arr[i].flops, "bytes": arr[i].bytes} for i in range(min(n.value, cap))]
