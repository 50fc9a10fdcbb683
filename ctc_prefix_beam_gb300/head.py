"""Thin Python binding of the label head (include/ctcpb.h): what produces the
decoder's ``log_prob`` and what trains it.

    y, mean, rstd = layer_norm(x, weight, bias)
    log_prob = log_probs(y, w, b)                       # [..., V] float32, for decode_offline / step_chunk
    loss, lse = cross_entropy(y, w, targets, b)         # the logits are never stored
    dy, dw, db = cross_entropy_backward(grad, y, w, targets, lse, b)
    dx, dweight, dbias = layer_norm_backward(dy, x, weight, mean, rstd)

Argument marshalling only, as in ``decoder``: tensors live on one CUDA device,
the calls run on its current stream and allocate their outputs and workspaces
from PyTorch unless they are given.  Rows are frames: ``x`` is [..., H].

What a call finds out on the device (a target out of range, a wait that gave up,
which makes its results invalid) is in the status word of its workspace.  A caller
that wants to know passes a workspace, and reads ``decoder.read_status(workspace)``
when it next waits for the GPU, before the workspace is used again.
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional

import torch

from . import decoder as D

NONE, MEAN, SUM = 0, 1, 2
DEV_TARGET = 0x20
_REDUCTIONS = {"none": NONE, "mean": MEAN, "sum": SUM}
_TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
_fns = None


def _lib():
    global _fns
    if _fns is None:
        L = D.lib()
        P, I, I64, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float
        SZ, SZP = ctypes.c_size_t, ctypes.POINTER(ctypes.c_size_t)
        sig = {
            "ctcpb_layer_norm": [I, I, P, I64, P, P, F, I64, I, P, I64, P, P, P],
            "ctcpb_layer_norm_workspace_size": [I64, I, SZP],
            "ctcpb_layer_norm_backward": [I, I, P, I64, P, I64, P, P, P, I64, I, P, I64, P, P, P, SZ, P],
            "ctcpb_log_probs_workspace_size": [I, I64, I, I, SZP],
            "ctcpb_log_probs": [I, I, P, I64, P, I64, P, I64, I, I, P, I64, P, SZ, P],
            "ctcpb_cross_entropy_workspace_size": [I, I64, I, I, I, SZP],
            "ctcpb_cross_entropy": [I, I, P, I64, P, I64, P, P, I64, I, I, I, I, P, P, P, SZ, P],
            "ctcpb_cross_entropy_backward": [I, I, P, P, I64, P, I64, P, P, P, I64, I, I, I, I, P, I64, P, I64, P, P, SZ,
                                             P],
        }
        fns = {}
        for name, args in sig.items():
            fn = getattr(L, name)
            fn.restype, fn.argtypes = I, args
            fns[name] = fn
        _fns = fns
    return _fns


def _rows(t: torch.Tensor, what: str, dtype=None):
    """``t`` [..., H] as rows: (tensor, N, H, row stride).  Leading dimensions
    that do not lie at one stride are copied together."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dim() < 1 or t.dtype not in _TYPES:
        raise ValueError(f"{what} must be a CUDA float32, bfloat16 or float16 tensor [..., H]")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{what} must be {dtype}")
    if t.is_contiguous():
        H = t.shape[-1]
        return t, t.numel() // H if H else 0, H, H
    if not (t.dim() == 2 and t.stride(1) == 1 and t.stride(0) >= t.shape[1]):
        H = t.shape[-1]
        ld = t.stride(-2) if t.dim() > 1 else H
        n = 1
        ok = (H <= 1 or t.stride(-1) == 1) and ld >= H
        for d in range(t.dim() - 2, -1, -1):
            ok = ok and (t.shape[d] <= 1 or t.stride(d) == ld * n)
            n *= t.shape[d]
        if not ok:
            t = t.contiguous()
    H = t.shape[-1]
    N = t.numel() // H if H else 0
    ld = t.stride(-2) if t.dim() > 1 and t.shape[-2] > 1 else H
    if N > 1 and t.dim() > 2 and t.shape[-2] == 1:  # the rows lie along an outer dimension
        ld = next(t.stride(d) for d in range(t.dim() - 3, -1, -1) if t.shape[d] > 1)
    return t, N, H, ld


def _matrix(w: torch.Tensor, H: int, dtype, device, what: str):
    """``w`` [V, H], rows at one stride: (tensor, V, row stride)."""
    if not isinstance(w, torch.Tensor) or w.dim() != 2 or w.dtype != dtype or w.device != device or w.shape[1] != H:
        raise ValueError(f"{what} must be a {dtype} tensor [V, {H}] on {device}")
    V = w.shape[0]
    if w.is_contiguous():
        return w, V, H
    if H > 1 and w.stride(1) != 1 or V > 1 and w.stride(0) < H:
        return w.contiguous(), V, H
    return w, V, w.stride(0) if V > 1 else H


def _params(dtype, n: int, device, first: str, p, second: str = "", q=None):
    """One or two parameter vectors (contiguous) and their type."""
    for name, v in ((first, p), (second, q)):
        if v is not None and (not isinstance(v, torch.Tensor) or v.shape != (n,) or v.device != device or
                              (v.dtype != dtype and v.dtype != torch.float32)):
            raise ValueError(f"{name} must be a {dtype} or float32 tensor [{n}] on {device}")
    if p is not None and q is not None and p.dtype != q.dtype:
        raise ValueError(f"{first} and {second} must be of one type")
    if p is not None and not p.is_contiguous():
        p = p.contiguous()
    if q is not None and not q.is_contiguous():
        q = q.contiguous()
    return p, q, dtype if p is None and q is None else (p if p is not None else q).dtype


def _given(t: torch.Tensor, shape, dtype, device, what: str) -> torch.Tensor:
    if not isinstance(t, torch.Tensor) or t.shape != shape or t.dtype != dtype or t.device != device \
            or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {dtype} tensor {list(shape)} on {device}")
    return t


@functools.lru_cache(maxsize=1024)
def _size(name: str, *args) -> int:
    n = ctypes.c_size_t()
    D._check(_lib()[name](*args, ctypes.byref(n)), name[6:])
    return n.value


def _workspace(ws, need: int, device):
    if ws is None:  # PyTorch's allocations start on 512-byte boundaries
        return torch.empty(need, dtype=torch.uint8, device=device), need
    return ws, D._check_buf(ws, need, device, "workspace")


def _p(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _raw_stream(dev: torch.device) -> int:
    return torch.cuda.current_stream(dev).cuda_stream


# the same without building a Stream object, where this PyTorch has it
_raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
if _raw is not None:
    def _raw_stream(dev: torch.device) -> int:  # noqa: F811
        return _raw(dev.index)


def _run(dev: torch.device, what: str, *args):
    """Call a library entry point on ``dev``'s current stream, ``dev`` current."""
    fn = _lib()[what]
    if dev.index == torch.cuda.current_device():
        rc = fn(*args, _raw_stream(dev))
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, _raw_stream(dev))
    if rc != D.OK:
        raise D.CtcpbError(rc, what[6:])


def layer_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None, *,
               eps: float = 1e-5, outputs=None):
    """Layer norm over the last dimension.  Returns (y like x, mean, rstd
    [...] float32); ``outputs``: the three to write."""
    xr, N, H, ldx = _rows(x, "x")
    dev, dt = xr.device, xr.dtype
    w, b, pt = _params(dt, H, dev, "weight", weight, "bias", bias)
    lead = x.shape[:-1]
    if outputs is None:
        y = torch.empty(x.shape, dtype=dt, device=dev)
        mean = torch.empty(lead, dtype=torch.float32, device=dev)
        rstd = torch.empty(lead, dtype=torch.float32, device=dev)
    else:
        y, mean, rstd = outputs
        _given(y, x.shape, dt, dev, "y")
        _given(mean, lead, torch.float32, dev, "mean")
        _given(rstd, lead, torch.float32, dev, "rstd")
    _run(dev, "ctcpb_layer_norm", _TYPES[dt], _TYPES[pt], _p(xr), ldx, _p(w), _p(b), eps, N, H, _p(y), H, _p(mean),
         _p(rstd))
    return y, mean, rstd


def layer_norm_workspace_size(N: int, H: int) -> int:
    return _size("ctcpb_layer_norm_workspace_size", N, H)


def layer_norm_backward(dy: torch.Tensor, x: torch.Tensor, weight: Optional[torch.Tensor], mean: torch.Tensor,
                        rstd: torch.Tensor, *, param_dtype=None, workspace: Optional[torch.Tensor] = None):
    """Gradients of ``layer_norm``: (dx like x, dweight, dbias [H]).  The last
    two are of ``weight``'s type, or ``param_dtype`` (x's) without a weight."""
    xr, N, H, ldx = _rows(x, "x")
    dev, dt = xr.device, xr.dtype
    dyr, n2, h2, lddy = _rows(dy, "dy", dt)
    if dy.shape != x.shape or dyr.device != dev:
        raise ValueError("dy must have x's shape and device")
    lead = x.shape[:-1]
    _given(mean, lead, torch.float32, dev, "mean")
    _given(rstd, lead, torch.float32, dev, "rstd")
    w, _, pt = _params(dt, H, dev, "weight", weight)
    if weight is None and param_dtype is not None:
        if param_dtype not in (dt, torch.float32):
            raise ValueError(f"param_dtype must be {dt} or float32")
        pt = param_dtype
    dx = torch.empty(x.shape, dtype=dt, device=dev)
    dw = torch.empty((H,), dtype=pt, device=dev)
    db = torch.empty((H,), dtype=pt, device=dev)
    ws, nbytes = _workspace(workspace, layer_norm_workspace_size(N, H), dev)
    _run(dev, "ctcpb_layer_norm_backward", _TYPES[dt], _TYPES[pt], _p(dyr), lddy, _p(xr), ldx, _p(w), _p(mean),
         _p(rstd), N, H, _p(dx), H, _p(dw), _p(db), _p(ws), nbytes)
    return dx, dw, db


def _head_args(x, weight, bias):
    xr, N, H, ldx = _rows(x, "x")
    dev, dt = xr.device, xr.dtype
    w, V, ldw = _matrix(weight, H, dt, dev, "weight")
    b, _, bt = _params(dt, V, dev, "bias", bias)
    return xr, N, H, ldx, dev, dt, w, V, ldw, b, bt


def log_probs_workspace_size(dtype, N: int, V: int, H: int) -> int:
    return _size("ctcpb_log_probs_workspace_size", _TYPES[dtype], N, V, H)


def log_probs(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None, *,
              out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The decoder's input, log_softmax(x weight^T + bias): float32 [..., V].
    x and weight are bfloat16 or float16.  ``out``: a tensor [..., V] to write,
    its rows at one stride (the padded rows of a wider tensor, for instance).
    ``workspace``'s status is 0 unless the results are invalid (CTCPB_DEV_TIMEOUT)."""
    xr, N, H, ldx, dev, dt, w, V, ldw, b, bt = _head_args(x, weight, bias)
    shape = (N, V) if x.dim() == 2 else (*x.shape[:-1], V)
    ldo = V
    if out is None:
        out = torch.empty(shape, dtype=torch.float32, device=dev)
    else:
        if not isinstance(out, torch.Tensor) or out.shape != shape or out.dtype != torch.float32 or out.device != dev:
            raise ValueError(f"out must be a float32 tensor {list(shape)} on {dev}")
        o, _, _, ldo = _rows(out, "out")
        if o is not out:
            raise ValueError("out's rows must lie at one stride, their labels contiguous")
    ws, nbytes = _workspace(workspace, log_probs_workspace_size(dt, N, V, H), dev)
    _run(dev, "ctcpb_log_probs", _TYPES[dt], _TYPES[bt], _p(xr), ldx, _p(w), ldw, _p(b), N, V, H, _p(out), ldo,
         _p(ws), nbytes)
    return out


def cross_entropy_workspace_size(dtype, N: int, V: int, H: int, backward: bool) -> int:
    return _size("ctcpb_cross_entropy_workspace_size", _TYPES[dtype], N, V, H, int(bool(backward)))


def _targets(targets, x, dev):
    if not isinstance(targets, torch.Tensor) or targets.dtype != torch.int32 or targets.device != dev or \
            targets.shape != x.shape[:-1]:
        raise ValueError(f"targets must be an int32 tensor {list(x.shape[:-1])} on {dev}")
    return targets.contiguous()


def _reduction(reduction: str) -> int:
    if reduction not in _REDUCTIONS:
        raise ValueError("reduction must be none, mean or sum")
    return _REDUCTIONS[reduction]


def _ignored(index: int) -> int:
    if not -2 ** 31 <= index < 2 ** 31:  # the C call would take its lowest 32 bits
        raise ValueError("ignore_index must be an int32 value")
    return index


def cross_entropy(x: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor, bias: Optional[torch.Tensor] = None, *,
                  ignore_index: int = -1, reduction: str = "mean", workspace: Optional[torch.Tensor] = None):
    """Softmax cross entropy of the logits x weight^T + bias, which are never
    stored.  ``targets`` int32 [...]; rows whose target is ``ignore_index`` take
    no part.  Returns (loss, lse [...]): float32, the loss a scalar or [...]
    (reduction "none").  ``D.read_status(workspace)`` holds ``DEV_TARGET`` if a
    target was out of range (such a row is ignored)."""
    xr, N, H, ldx, dev, dt, w, V, ldw, b, bt = _head_args(x, weight, bias)
    t, red = _targets(targets, x, dev), _reduction(reduction)
    lead = x.shape[:-1]
    loss = torch.empty(lead if red == NONE else (), dtype=torch.float32, device=dev)
    lse = torch.empty(lead, dtype=torch.float32, device=dev)
    ws, nbytes = _workspace(workspace, cross_entropy_workspace_size(dt, N, V, H, False), dev)
    _run(dev, "ctcpb_cross_entropy", _TYPES[dt], _TYPES[bt], _p(xr), ldx, _p(w), ldw, _p(b), _p(t), N, V, H,
         _ignored(ignore_index), red, _p(loss), _p(lse), _p(ws), nbytes)
    return loss, lse


def cross_entropy_backward(grad: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor,
                           lse: torch.Tensor, bias: Optional[torch.Tensor] = None, *, ignore_index: int = -1,
                           reduction: str = "mean", workspace: Optional[torch.Tensor] = None):
    """Gradients of ``cross_entropy`` for the loss's gradient ``grad`` (float32,
    a scalar, or [...] for reduction "none"): (dx like x, dweight, dbias; dbias
    is None without a bias).  ``workspace``'s status is as ``cross_entropy``'s."""
    xr, N, H, ldx, dev, dt, w, V, ldw, b, bt = _head_args(x, weight, bias)
    t, red = _targets(targets, x, dev), _reduction(reduction)
    lead = x.shape[:-1]
    _given(lse, lead, torch.float32, dev, "lse")
    _given(grad, lead if red == NONE else (), torch.float32, dev, "grad")
    dx = torch.empty(x.shape, dtype=dt, device=dev)
    dw = torch.empty((V, H), dtype=dt, device=dev)
    db = torch.empty((V,), dtype=bt, device=dev) if bias is not None else None
    ws, nbytes = _workspace(workspace, cross_entropy_workspace_size(dt, N, V, H, True), dev)
    _run(dev, "ctcpb_cross_entropy_backward", _TYPES[dt], _TYPES[bt], _p(grad), _p(xr), ldx, _p(w), ldw, _p(b),
         _p(t), _p(lse), N, V, H, _ignored(ignore_index), red, _p(dx), H, _p(dw), H, _p(db), _p(ws), nbytes)
    return dx, dw, db
