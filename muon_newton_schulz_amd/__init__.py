"""MI355X (gfx950) Muon / Newton-Schulz / Gram-NS / NorMuon / Dion3 optimizer step.

Thin Python binding over the C ABI in include/muon_ns.h: it turns torch tensors into
device pointers and sizes and calls the HIP library; every step of the computation runs in
the library's kernels. PyTorch supplies device memory and the current stream only. The
library must be built (``python -m muon_newton_schulz_amd.build``); there is no fallback.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import struct
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
           "grouped_linear", "grouped_input_grad", "grouped_bias_grad",
           "expert_order", "balance_loss", "grad_norm", "clip_grad_norm",
           "step_workspace_size", "ns_workspace_size", "normuon_workspace_size",
           "restart_mask", "profile_begin", "profile_set_flush", "profile_end", "MnsError",
           "load"]

_ACTIVATIONS = {None: _abi.MNS_ACT_NONE, "relu": _abi.MNS_ACT_RELU, "relu2": _abi.MNS_ACT_RELU2,
                "gelu": _abi.MNS_ACT_GELU, "silu": _abi.MNS_ACT_SILU}
_STORAGE = {torch.bfloat16: MNS_BF16, torch.float32: MNS_F32}
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
            if device.index != torch._C._cuda_getDevice():
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
    if t.is_contiguous():
        return cols
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


def _one_gpu(first: torch.Tensor, others, what: str) -> torch.device:
    """_on_one_gpu of tensors that are rarely elsewhere: compares device numbers (-1: not a GPU)."""
    index = first.get_device()
    if index >= 0:
        for t in others:
            if t is not None and t.get_device() != index:
                break
        else:
            return first.device
    return _on_one_gpu([first, *others], what)


def _check_offsets(offsets: torch.Tensor, groups: int, what: str) -> None:
    if offsets.dtype != torch.int64 or offsets.shape != (groups + 1,) or not offsets.is_contiguous():
        raise ValueError(f"{what}: offsets must be contiguous int64 of shape ({groups + 1},)")


@functools.lru_cache(maxsize=4096)
def _size_query(name: str, *args) -> int:
    """Bytes a workspace query of the library answers: a function of its arguments alone, so asked once
    for each."""
    need = ctypes.c_size_t(0)
    check(getattr(load(), name)(*args, ctypes.byref(need)), name)
    return need.value


def _optional_workspace(nbytes: int, dev, workspace):
    """(tensor, pointer, bytes) of a call's workspace, nothing for a call without one."""
    if nbytes == 0:
        return None, None, 0
    ws = _workspace(nbytes, dev, workspace)
    return ws, ws.data_ptr(), ws.numel() * ws.element_size()


def _activation(activation, what: str) -> int:
    if activation not in _ACTIVATIONS:
        names = sorted(a for a in _ACTIVATIONS if a)
        raise ValueError(f"{what}: activation must be None or one of {names}")
    return _ACTIVATIONS[activation]


def _rowwise(t: torch.Tensor | None, name: str, shape, dtype, what: str) -> int:
    """Row pitch of an optional 2-D tensor of the given shape and dtype (0 for None)."""
    if t is None:
        return 0
    if t.shape != shape or t.dtype != dtype:
        raise ValueError(f"{what}: {name} must be {shape} {dtype}, got {tuple(t.shape)} {t.dtype}")
    return _pitch(t, name, what)


def _itself_or_apart(out, name: str, same, others, what: str) -> None:
    """`out` may be one of `same` (its memory and pitch) and otherwise overlap nothing."""
    if out is None:
        return
    for other_name, t in others:
        if t is not None and not _apart(out, t):
            raise ValueError(f"{what}: {name} may not overlap {other_name}")
    for other_name, t in same:
        if t is None or _apart(out, t):
            continue
        if t.data_ptr() != out.data_ptr() or t.stride() != out.stride():
            raise ValueError(f"{what}: {name} must be {other_name} itself or lie apart from it")


def _ptr_or_none(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


def _layer_operands(A, W, transpose_w: bool, a_name: str, what: str):
    """Checks of a layer's rows and weights: dtype code, (groups, n, k), rows, pitch, output width."""
    code = _dtype_code(A)
    if W.dim() != 3:
        raise ValueError(f"{what}: W must be 3-D (experts, n, k)")
    if W.dtype != A.dtype:
        raise TypeError(f"{what}: {a_name} and W must share one storage dtype "
                        f"({a_name} {A.dtype}, W {W.dtype})")
    groups, n, k = W.shape
    inner, width = (n, k) if transpose_w else (k, n)
    if A.dim() != 2 or A.shape[1] != inner:
        raise ValueError(f"{what}: {a_name} must be 2-D with rows of {inner}, got {tuple(A.shape)}")
    if not W.is_contiguous():
        raise ValueError(f"{what}: W must be contiguous")
    return code, groups, n, k, A.shape[0], _pitch(A, a_name, what), width


def _new_rows(rows: int, width: int, like: torch.Tensor, zeros: bool) -> torch.Tensor:
    """A new row-wise output; zeros when the call's own filling of unowned rows is off."""
    if zeros:
        return like.new_zeros((rows, width))
    if like.shape[1] == width and like.is_contiguous():
        return torch.empty_like(like)
    return like.new_empty((rows, width))


def grouped_linear(X: torch.Tensor, W: torch.Tensor, offsets: torch.Tensor, *,
                   bias: torch.Tensor | None = None, activation: str | None = None,
                   residual: torch.Tensor | None = None, keep_z: bool = False,
                   out: torch.Tensor | None = None, out_z: torch.Tensor | None = None,
                   workspace: torch.Tensor | None = None, stream=None):
    """A layer of experts in one product: Z_e = X_e W_e^T + bias_e, Y = act(Z) + residual, rows sorted
    by expert as in grouped_matmul (a plain layer is a stack of one). Returns Y, or with an
    activation and ``keep_z`` (or a given ``out_z``) (Y, Z): Z is what grouped_input_grad and
    grouped_bias_grad take.

    bias: contiguous (experts, n); residual, ``out``, ``out_z``: (rows, n) at any row pitch, ``out`` may
    be the residual itself; all of X's dtype. activation: None, "relu", "relu2" (relu squared), "gelu"
    (z Phi(z)) or "silu". Between the product and each output's one rounding everything is float32; gelu
    of bfloat16 layers, and its slope in the gradients, is a fit within 1.5e-5 of the normal tail's mass
    (|z| up to 5; in full in muon_ns.h).
    Rows that belong to no expert come back as zeros in new outputs and are left as they are in given
    ones. Autograd does not see the call."""
    what = "grouped_linear"
    code, groups, n, k, rows, ldx, _ = _layer_operands(X, W, False, "X", what)
    act = _activation(activation, what)
    keep_z = keep_z or out_z is not None
    if keep_z and activation is None:
        raise ValueError(f"{what}: without an activation no gradient needs Z")
    if bias is not None:
        if bias.shape != (groups, n) or bias.dtype != X.dtype:
            raise ValueError(f"{what}: bias must be {(groups, n)} {X.dtype}, "
                             f"got {tuple(bias.shape)} {bias.dtype}")
        if not bias.is_contiguous():
            raise ValueError(f"{what}: bias must be contiguous")
    ldr = _rowwise(residual, "residual", (rows, n), X.dtype, what)
    ldy = _rowwise(out, "out", (rows, n), X.dtype, what)
    ldz = _rowwise(out_z, "out_z", (rows, n), X.dtype, what)
    if out is not None or out_z is not None:
        others = [("X", X), ("W", W), ("bias", bias), ("offsets", offsets)]
        _itself_or_apart(out, "out", [("residual", residual)], others + [("out_z", out_z)], what)
        _itself_or_apart(out_z, "out_z", [], others + [("residual", residual)], what)
    _check_offsets(offsets, groups, what)
    dev = _one_gpu(X, (W, bias, residual, out, out_z, offsets), what)
    with _OnStream(dev, stream) as handle:
        fill = out is None and out_z is None        # else what is new is made of zeros
        Y, Z = out, out_z
        if Y is None:
            Y, ldy = _new_rows(rows, n, X, not fill), n
        if keep_z and Z is None:
            Z, ldz = _new_rows(rows, n, X, not fill), n
        keep, ws, nbytes = _optional_workspace(
            _size_query("mns_grouped_layer_workspace_size", 0, code, groups, rows, n, k), dev, workspace)
        check(load().grouped_linear(X.data_ptr(), ldx, W.data_ptr(), _ptr_or_none(bias), act,
                                    _ptr_or_none(residual), ldr, _ptr_or_none(Z), ldz, Y.data_ptr(),
                                    ldy, code, offsets.data_ptr(), groups, rows, n, k, int(fill), ws,
                                    nbytes, handle), what)
    return (Y, Z) if keep_z else Y


def grouped_input_grad(dY: torch.Tensor, W: torch.Tensor, offsets: torch.Tensor, *,
                       activation: str | None = None, Z: torch.Tensor | None = None,
                       residual: torch.Tensor | None = None, out: torch.Tensor | None = None,
                       workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Gradient of a layer's input: dX_e = (dY_e W_e) act'(Z) + residual. ``activation`` and ``Z`` are
    those of the layer that produced the input (then dX is the gradient of that layer's Z); ``residual``
    is a gradient that reaches the input past this layer. Z, residual and ``out``: (rows, k) at any row
    pitch; ``out`` may be Z or the residual itself. relu's slope at 0 is 0. Rows that belong to no
    expert as in grouped_matmul. Autograd does not see the call."""
    what = "grouped_input_grad"
    code, groups, n, k, rows, lddy, _ = _layer_operands(dY, W, True, "dY", what)
    act = _activation(activation, what)
    if (Z is None) != (activation is None):
        raise ValueError(f"{what}: activation and Z go together")
    ldz = _rowwise(Z, "Z", (rows, k), dY.dtype, what)
    ldr = _rowwise(residual, "residual", (rows, k), dY.dtype, what)
    lddx = _rowwise(out, "out", (rows, k), dY.dtype, what)
    _itself_or_apart(out, "out", [("Z", Z), ("residual", residual)],
                     [("dY", dY), ("W", W), ("offsets", offsets)], what)
    _check_offsets(offsets, groups, what)
    dev = _one_gpu(dY, (W, Z, residual, out, offsets), what)
    with _OnStream(dev, stream) as handle:
        dX = out
        if dX is None:
            dX, lddx = _new_rows(rows, k, dY, False), k
        keep, ws, nbytes = _optional_workspace(
            _size_query("mns_grouped_layer_workspace_size", 1, code, groups, rows, n, k), dev, workspace)
        check(load().grouped_input_grad(dY.data_ptr(), lddy, W.data_ptr(), act, _ptr_or_none(Z), ldz,
                                        _ptr_or_none(residual), ldr, dX.data_ptr(), lddx, code,
                                        offsets.data_ptr(), groups, rows, n, k, int(out is None), ws,
                                        nbytes, handle), what)
    return dX


def grouped_bias_grad(dY: torch.Tensor, offsets: torch.Tensor, *, activation: str | None = None,
                      Z: torch.Tensor | None = None, out: torch.Tensor | None = None,
                      out_dtype: torch.dtype | None = None, out_dz: torch.Tensor | None = None,
                      workspace: torch.Tensor | None = None, stream=None):
    """Gradient of a layer's bias, db_e = the sum of expert e's rows of dZ = dY act'(Z), as (experts, n).
    With an activation returns (db, dZ), else db (dZ is dY). dY, Z and ``out_dz``: (rows, n) at any row
    pitch, ``out_dz`` may be dY or Z itself; db is of ``out``'s dtype, else ``out_dtype``, else dY's
    (dY's or float32; the sums are float32 and of the unrounded products). Rows that belong to no
    expert as in grouped_matmul. Autograd does not see the call."""
    what = "grouped_bias_grad"
    code = _dtype_code(dY)
    act = _activation(activation, what)
    if dY.dim() != 2:
        raise ValueError(f"{what}: dY must be 2-D (rows x width)")
    if offsets.dim() != 1 or offsets.shape[0] < 2:
        raise ValueError(f"{what}: offsets must hold at least two entries")
    if (Z is None) != (activation is None):
        raise ValueError(f"{what}: activation and Z go together")
    if out_dz is not None and activation is None:
        raise ValueError(f"{what}: without an activation dZ is dY, and out_dz is not written")
    rows, n, groups = dY.shape[0], dY.shape[1], offsets.shape[0] - 1
    lddy = _pitch(dY, "dY", what)
    ldz = _rowwise(Z, "Z", (rows, n), dY.dtype, what)
    lddz = _rowwise(out_dz, "out_dz", (rows, n), dY.dtype, what)
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else dY.dtype
    if out_dtype not in (dY.dtype, torch.float32):
        raise TypeError(f"{what}: the output must be {dY.dtype} or float32, not {out_dtype}")
    if out is not None:
        if tuple(out.shape) != (groups, n) or out.dtype != out_dtype:
            raise ValueError(f"{what}: out must be {(groups, n)} {out_dtype}, "
                             f"got {tuple(out.shape)} {out.dtype}")
        if not out.is_contiguous():
            raise ValueError(f"{what}: out must be contiguous")
    _itself_or_apart(out, "out", [], [("dY", dY), ("Z", Z), ("out_dz", out_dz),
                                      ("offsets", offsets)], what)
    _itself_or_apart(out_dz, "out_dz", [("dY", dY), ("Z", Z)], [("offsets", offsets)], what)
    _check_offsets(offsets, groups, what)
    dev = _one_gpu(dY, (Z, out, out_dz, offsets), what)
    need = _size_query("mns_grouped_bias_grad_workspace_size", groups, rows, n)
    with _OnStream(dev, stream) as handle:
        db = dY.new_empty((groups, n), dtype=out_dtype) if out is None else out
        dZ = out_dz
        if activation is not None and dZ is None:
            dZ, lddz = _new_rows(rows, n, dY, False), n
        keep, ws, nbytes = _optional_workspace(need, dev, workspace)
        check(load().grouped_bias_grad(dY.data_ptr(), lddy, act, _ptr_or_none(Z), ldz,
                                       _ptr_or_none(dZ), lddz, code, offsets.data_ptr(), groups, rows,
                                       n, db.data_ptr(),
                                       MNS_F32 if out_dtype == torch.float32 else MNS_BF16,
                                       int(out_dz is None), ws, nbytes, handle), what)
    return db if activation is None else (db, dZ)


def _ids(expert_ids: torch.Tensor, what: str) -> None:
    if expert_ids.dtype != torch.int64 or not expert_ids.is_contiguous():
        raise ValueError(f"{what}: expert_ids must be a contiguous int64 tensor")


def expert_order(expert_ids: torch.Tensor, experts: int, *, order: bool = True,
                 workspace: torch.Tensor | None = None, stream=None):
    """A router's assignments by expert: (counts, offsets, order), int64 on the GPU, nothing read by the
    host. expert_ids: int64, any shape ((tokens, top) as torch.topk gives it), contiguous; a value outside
    0 .. experts - 1, such as -1 for a padded token, is an assignment to no expert. counts: (experts,).
    offsets: (experts + 1,), what the grouped calls take. order: the flat indices of the assignments by
    expert, each expert's in their own order, those of no expert last, so ``X[order // top]`` are the rows
    the grouped calls take (None with ``order=False``). At most 2048 experts."""
    what = "expert_order"
    _ids(expert_ids, what)
    dev = _one_gpu(expert_ids, (), what)
    m = expert_ids.numel()
    need = _size_query("mns_expert_order_workspace_size", m, experts)
    with _OnStream(dev, stream) as handle:
        counts, offsets = expert_ids.new_empty(experts), expert_ids.new_empty(experts + 1)
        places = expert_ids.new_empty(m) if order else None
        keep, ws, nbytes = _optional_workspace(need, dev, workspace)
        check(load().expert_order(expert_ids.data_ptr(), m, experts, counts.data_ptr(),
                                  offsets.data_ptr(), _ptr_or_none(places), ws, nbytes, handle), what)
    return counts, offsets, places


def balance_loss(logits: torch.Tensor, expert_ids: torch.Tensor, counts: torch.Tensor, *,
                 scale: float = 1.0, grad: bool = True, out: torch.Tensor | None = None,
                 workspace: torch.Tensor | None = None, stream=None):
    """The balance loss of a router and its gradient: (loss, dlogits), loss a float32 scalar tensor.

    loss = scale E sum_e f_e P_e, with f_e = counts_e / N expert e's share of the N assignments and P_e the
    mean of softmax(logits)_e over the assigned tokens, each weighted by its assignments; dlogits is its
    gradient (f is taken as constant), for an upstream gradient of 1: ``scale`` takes any other. logits:
    (tokens, E) float32 or bfloat16 at any row pitch; expert_ids: (tokens, top) int64; counts: (E,) int64,
    expert_order's. A token without an assignment adds nothing and gets zeros, whatever its logits hold, and
    so does one whose logits are all -inf. dlogits has the logits' dtype: a new tensor, ``out`` (may be the
    logits themselves), or None with ``grad=False``. Autograd does not see the call."""
    what = "balance_loss"
    code = _dtype_code(logits)
    if logits.dim() != 2 or expert_ids.dim() != 2 or expert_ids.shape[0] != logits.shape[0]:
        raise ValueError(f"{what}: logits must be (tokens, experts) and expert_ids (tokens, top)")
    _ids(expert_ids, what)
    tokens, experts = logits.shape
    if counts.dtype != torch.int64 or counts.shape != (experts,) or not counts.is_contiguous():
        raise ValueError(f"{what}: counts must be contiguous int64 of shape ({experts},)")
    if out is not None and not grad:
        raise ValueError(f"{what}: out without a gradient")
    ldl = _pitch(logits, "logits", what)
    ldd = _rowwise(out, "out", (tokens, experts), logits.dtype, what)
    _itself_or_apart(out, "out", [("logits", logits)],
                     [("expert_ids", expert_ids), ("counts", counts)], what)
    dev = _one_gpu(logits, (expert_ids, counts, out), what)
    need = _size_query("mns_balance_workspace_size", tokens, experts)
    with _OnStream(dev, stream) as handle:
        loss = torch.empty((), dtype=torch.float32, device=dev)
        dlogits = out
        if grad and dlogits is None:
            dlogits, ldd = _new_rows(tokens, experts, logits, False), experts
        keep, ws, nbytes = _optional_workspace(need, dev, workspace)
        check(load().balance_loss(logits.data_ptr(), ldl, code, expert_ids.data_ptr(),
                                  expert_ids.shape[1], counts.data_ptr(), tokens, experts, scale,
                                  loss.data_ptr(), _ptr_or_none(dlogits), ldd, ws, nbytes, handle),
              what)
    return loss, dlogits


def _tensor_list(grads, out, what: str):
    grads = _as_list(grads)
    if not grads:
        raise ValueError(f"{what}: no gradients")
    outs = grads if out is None else _as_list(out)
    if len(outs) != len(grads):
        raise ValueError(f"{what}: out must hold as many tensors as grads")
    dev = grads[0].device
    index, codes, flat = dev.index, _STORAGE, []
    for i, g in enumerate(grads):             # few reads a tensor: lists are long
        code = codes.get(g.dtype)
        if code is None:
            _dtype_code(g)
        if not g.is_contiguous():
            raise ValueError(f"{what}: gradient {i} must be contiguous")
        if g.get_device() != index:           # -1 is not a GPU, whose index is None
            _on_one_gpu(grads + outs, what)
        at = to = g.data_ptr()
        if outs is not grads and outs[i] is not g:
            o = outs[i]
            if o.shape != g.shape or o.dtype != g.dtype or not o.is_contiguous():
                raise ValueError(f"{what}: out {i} must match its gradient and be contiguous")
            if o.get_device() != index:
                _on_one_gpu(grads + outs, what)
            to = o.data_ptr()
        flat += (at, to, g.numel(), code)
    return struct.pack("QQqi4x" * len(grads), *flat), len(grads), dev


def grad_norm(grads, *, workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The global norm over one gradient or a list of them (contiguous, float32 or bfloat16 in any
    mixture, any shapes): sqrt of the sum of every element's square, summed in float64, as a float32
    scalar tensor. Nothing is read by the host."""
    what = "grad_norm"
    arr, count, dev = _tensor_list(grads, None, what)
    with _OnStream(dev, stream) as handle:
        norm = torch.empty((), dtype=torch.float32, device=dev)
        ws = _workspace(_size_query("mns_clip_workspace_size", count), dev, workspace)
        check(load().grad_norm(arr, count, norm.data_ptr(), ws.data_ptr(),
                               ws.numel() * ws.element_size(), handle), what)
    return norm


def clip_grad_norm(grads, max_norm: float, *, eps: float = 1e-6, out=None,
                   workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Scales gradients by min(1, max_norm / (norm + eps)), norm their global norm (grad_norm), which is
    returned: the step before muon_step. In place, or into ``out`` (a tensor, or a list of them, like the
    gradients). A NaN norm makes every gradient NaN, an infinite one makes finite gradients 0. No output may
    overlap another one or another gradient, so no gradient may be listed twice."""
    what = "clip_grad_norm"
    arr, count, dev = _tensor_list(grads, out, what)
    with _OnStream(dev, stream) as handle:
        norm = torch.empty((), dtype=torch.float32, device=dev)
        ws = _workspace(_size_query("mns_clip_workspace_size", count), dev, workspace)
        check(load().clip_grad_norm(arr, count, max_norm, eps, norm.data_ptr(), ws.data_ptr(),
                                    ws.numel() * ws.element_size(), handle), what)
    return norm


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
