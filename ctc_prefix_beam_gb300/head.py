"""Thin Python binding of the label head (include/ctcpb.h): what produces the
decoder's ``log_prob`` and what trains it.

    y, mean, rstd = layer_norm(x, weight, bias)
    log_prob = log_probs(y, w, b)                       # [..., V] float32, for decode_offline / step_chunk
    loss, lse = cross_entropy(y, w, targets, b)         # the logits are never stored
    dy, dw, db = cross_entropy_backward(grad, y, w, targets, lse, b)
    dx, dweight, dbias = layer_norm_backward(dy, x, weight, mean, rstd)

Around it: a norm for convolutional blocks, dropout, and the losses that train the
model from the decoder's own N-best lists (tokens [B, N, L] and their lengths):

    y, mean, rstd = group_norm(x, groups, weight, bias, lengths=lengths, activation="silu")
    y = dropout(x, p, rng, residual=r)                  # rng: int64 [2] on the device, (seed, offset)
    nll, lse = cross_entropy(y, w, tokens, b, reduction="none")
    loss, stats, dnll = policy_loss(nll, old_nll, advantages, lengths=lengths, ref_nll=ref_nll, kl_weight=k, grad=one)
    loss, margins, dnll = preference_loss(nll, chosen, rejected, lengths=lengths, ref_nll=ref_nll, grad=one)
    dy, dw, db = cross_entropy_backward(dnll, y, w, tokens, lse, b, reduction="none")

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

NONE, MEAN, SUM, SEQUENCE_MEAN = 0, 1, 2, 3
DEV_TARGET = 0x20
_REDUCTIONS = {"none": NONE, "mean": MEAN, "sum": SUM}
_SEQ_REDUCTIONS = {**_REDUCTIONS, "sequence_mean": SEQUENCE_MEAN}
_ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2}
_TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
_fns = None


def _lib():
    global _fns
    if _fns is None:
        L = D.lib()
        P, I, I64, F, DBL = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_double
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
            "ctcpb_group_norm": [I, I, P, I64, I64, P, P, P, F, I, I, I, I, I, P, I64, I64, P, P, P, SZ, P],
            "ctcpb_group_norm_workspace_size": [I, I, I, I, I, I, SZP],
            "ctcpb_group_norm_backward": [I, I, P, I64, I64, P, I64, I64, P, P, P, P, P, I, I, I, I, I, P, I64, I64, P, P, P,
                                          SZ, P],
            "ctcpb_dropout": [I, P, I64, P, I64, DBL, P, I64, I, P, I64, P],
            "ctcpb_policy_loss_workspace_size": [I64, I64, SZP],
            "ctcpb_policy_loss": [P, I64, P, I64, P, I64, P, I64, P, I64, I64, DBL, DBL, F, I, P, P, P, P, P, SZ, P],
            "ctcpb_preference_loss_workspace_size": [I64, I, I64, SZP],
            "ctcpb_preference_loss": [P, I64, P, I64, P, P, P, I64, I, I64, F, F, F, I, I, P, P, P, P, P, SZ, P],
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
    if need == 0:
        return None, 0
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


_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)  # without its lazy initialisation


def _run(dev: torch.device, what: str, *args):
    """Call a library entry point on ``dev``'s current stream, ``dev`` current."""
    fn = (_fns or _lib())[what]
    if dev.index == _current_device():
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


def _like(t: torch.Tensor) -> torch.Tensor:
    """A contiguous tensor of t's shape, type and device."""
    return torch.empty_like(t) if t.is_contiguous() else torch.empty(t.shape, dtype=t.dtype, device=t.device)


def _frames(t: torch.Tensor, what: str, dtype=None):
    """``t`` [B, T, C], channels contiguous and the rows of an utterance at one
    stride of at least C (else it is copied): (tensor, its strides)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dim() != 3 or t.dtype not in _TYPES:
        raise ValueError(f"{what} must be a CUDA float32, bfloat16 or float16 tensor [B, T, C]")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{what} must be {dtype}")
    B, T, C = t.shape
    if t.is_contiguous():
        return t, T * C, C
    if C > 1 and t.stride(2) != 1 or T > 1 and t.stride(1) < C:
        t = t.contiguous()
    return t, t.stride(0) if B > 1 else T * C, t.stride(1) if T > 1 else C


def _ints(t, shape, device, what: str):
    """An optional int32 tensor (contiguous)."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.dtype != torch.int32 or t.device != device or t.shape != shape:
        raise ValueError(f"{what} must be an int32 tensor {list(shape)} on {device}")
    return t if t.is_contiguous() else t.contiguous()


def _activation(name: str) -> int:
    if name not in _ACTIVATIONS:
        raise ValueError("activation must be none, relu or silu")
    return _ACTIVATIONS[name]


def _groups(groups: int, C: int) -> int:
    if not isinstance(groups, int) or groups < 1 or C < 1 or C % groups:
        raise ValueError(f"groups must divide the {C} channels")
    return groups


def group_norm(x: torch.Tensor, groups: int, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
               *, lengths: Optional[torch.Tensor] = None, eps: float = 1e-5, activation: str = "none", outputs=None,
               workspace: Optional[torch.Tensor] = None):
    """Group norm and an activation (none, relu, silu) over channels-last frames
    [B, T, C]: a group's statistics are over its channels and an utterance's first
    ``lengths[b]`` (int32 [B]) frames; later frames are not read, and y is 0 there.
    Returns (y like x, mean, rstd [B, groups] float32); ``outputs``: the three to
    write (y may not be x)."""
    act = _activation(activation)
    xr, sb, st = _frames(x, "x")
    B, T, C = x.shape
    G, dev, dt = _groups(groups, C), xr.device, xr.dtype
    w, b, pt = _params(dt, C, dev, "weight", weight, "bias", bias)
    n = _ints(lengths, (B,), dev, "lengths")
    if outputs is None:
        y = _like(xr)
        mean = torch.empty((B, G), dtype=torch.float32, device=dev)
        rstd = torch.empty_like(mean)
    else:
        y, mean, rstd = outputs
        _given(y, x.shape, dt, dev, "y")
        _given(mean, (B, G), torch.float32, dev, "mean")
        _given(rstd, (B, G), torch.float32, dev, "rstd")
        if y.data_ptr() == xr.data_ptr() and y.numel():
            raise ValueError("y must not be x")
    ws, nbytes = _workspace(workspace, group_norm_workspace_size(dt, B, T, C, G, False), dev)
    _run(dev, "ctcpb_group_norm", _TYPES[dt], _TYPES[pt], xr.data_ptr(), sb, st, _p(w), _p(b), _p(n), eps, act, B, T, C, G,
         y.data_ptr(), T * C, C, mean.data_ptr(), rstd.data_ptr(), _p(ws), nbytes)
    return y, mean, rstd


def group_norm_workspace_size(dtype, B: int, T: int, C: int, groups: int, backward: bool) -> int:
    return _size("ctcpb_group_norm_workspace_size", _TYPES[dtype], B, T, C, groups, int(bool(backward)))


def group_norm_backward(dy: torch.Tensor, x: torch.Tensor, groups: int, weight: Optional[torch.Tensor],
                        bias: Optional[torch.Tensor], mean: torch.Tensor, rstd: torch.Tensor, *,
                        lengths: Optional[torch.Tensor] = None, activation: str = "none", param_dtype=None,
                        workspace: Optional[torch.Tensor] = None):
    """Gradients of ``group_norm`` (the same weight, bias, lengths and activation):
    (dx like x, dweight, dbias [C]).  The last two are of the parameters' type, or
    ``param_dtype`` (x's) without any."""
    act = _activation(activation)
    xr, sb, st = _frames(x, "x")
    B, T, C = x.shape
    G, dev, dt = _groups(groups, C), xr.device, xr.dtype
    dyr, db_, dt_ = _frames(dy, "dy", dt)
    if dy.shape != x.shape or dyr.device != dev:
        raise ValueError("dy must have x's shape and device")
    _given(mean, (B, G), torch.float32, dev, "mean")
    _given(rstd, (B, G), torch.float32, dev, "rstd")
    w, b, pt = _params(dt, C, dev, "weight", weight, "bias", bias)
    if weight is None and bias is None and param_dtype is not None:
        if param_dtype not in (dt, torch.float32):
            raise ValueError(f"param_dtype must be {dt} or float32")
        pt = param_dtype
    n = _ints(lengths, (B,), dev, "lengths")
    dx = _like(xr)
    dw = torch.empty((C,), dtype=pt, device=dev)
    db = torch.empty_like(dw)
    ws, nbytes = _workspace(workspace, group_norm_workspace_size(dt, B, T, C, G, True), dev)
    _run(dev, "ctcpb_group_norm_backward", _TYPES[dt], _TYPES[pt], dyr.data_ptr(), db_, dt_, xr.data_ptr(), sb, st, _p(w), _p(b),
         _p(n), mean.data_ptr(), rstd.data_ptr(), act, B, T, C, G, dx.data_ptr(), T * C, C, dw.data_ptr(), db.data_ptr(), _p(ws),
         nbytes)
    return dx, dw, db


_TWO = torch.Size((2,))


def dropout(x: torch.Tensor, p: float, rng: torch.Tensor, *, residual: Optional[torch.Tensor] = None,
            out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Dropout of x [..., H] with probability ``p`` (held to 2^-16), what is kept
    scaled up, added to ``residual`` if there is one.  Whether an element is kept
    is a function of its index in x's shape and of ``rng``, an int64 tensor [2] on
    x's device that holds a seed and an offset; the call does not change it.
    ``out``: the tensor to write, which may be x or residual."""
    xr, N, H, ldx = _rows(x, "x")
    dev, dt = xr.device, xr.dtype
    if not isinstance(rng, torch.Tensor) or rng.dtype is not torch.int64 or rng.shape != _TWO or rng.device != dev or \
            not rng.is_contiguous():
        raise ValueError(f"rng must be a contiguous int64 tensor [2] on {dev}")
    r, ldr = None, 0
    if residual is not None:
        r, _, _, ldr = _rows(residual, "residual", dt)
        if residual.shape != x.shape or r.device != dev:
            raise ValueError("residual must have x's shape and device")
    y = _like(x) if out is None else _given(out, x.shape, dt, dev, "out")
    _run(dev, "ctcpb_dropout", _TYPES[dt], xr.data_ptr(), ldx, _p(r), ldr, p, rng.data_ptr(), N, H, y.data_ptr(), H)
    return y


def dropout_backward(dy: torch.Tensor, p: float, rng: torch.Tensor, *, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The gradient of ``dropout`` with respect to x (the residual's is dy): the
    same elements, for the same ``rng``, kept and scaled."""
    return dropout(dy, p, rng, out=out)


def _scores(t, shape, device, what: str):
    """float32 rows [..., L] at one stride: (tensor, stride)."""
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.float32 or t.shape != shape or t.device != device:
        raise ValueError(f"{what} must be a float32 tensor {list(shape)} on {device}")
    if t.is_contiguous():
        return t, shape[-1]
    t, _, _, ld = _rows(t, what)
    return t, ld


def _loss_grad(grad, reduction: int, shape, device):
    if grad is not None:
        _given(grad, shape if reduction == NONE else (), torch.float32, device, "grad")
    return grad


def _status_or(workspace, need: int, device):
    """A loss's workspace: small calls have only the status in it, and do without."""
    return (None, 0) if workspace is None and need <= 256 else _workspace(workspace, need, device)


def policy_loss_workspace_size(S: int, L: int) -> int:
    return _size("ctcpb_policy_loss_workspace_size", S, L)


def policy_loss(nll: torch.Tensor, old_nll: torch.Tensor, advantages: torch.Tensor, *,
                lengths: Optional[torch.Tensor] = None, ref_nll: Optional[torch.Tensor] = None, clip_low: float = 0.2,
                clip_high: float = 0.2, kl_weight: float = 0.0, reduction: str = "mean",
                grad: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """The clipped policy loss of sequences of tokens, whose negative
    log-probabilities ``nll`` [..., L] are ``cross_entropy``'s losses (reduction
    "none"), with the KL term of ``ref_nll``.  ``old_nll`` is of the model that made
    the sequences; ``advantages`` float32 [...], or [..., L] for each token;
    ``lengths`` int32 [...].  ``reduction``: none ([..., L]), mean (over all tokens),
    sum, or sequence_mean (the mean over sequences of each one's mean).  Returns
    (loss, stats), stats float32 [2] the mean KL and the share of clipped tokens;
    with the loss's gradient ``grad`` (float32, a scalar or [..., L]), known when
    the loss is made, (loss, stats, dnll): ``cross_entropy_backward``'s grad."""
    if reduction not in _SEQ_REDUCTIONS:
        raise ValueError("reduction must be none, mean, sum or sequence_mean")
    red = _SEQ_REDUCTIONS[reduction]
    if not isinstance(nll, torch.Tensor) or not nll.is_cuda or nll.dim() < 1:
        raise ValueError("nll must be a CUDA float32 tensor [..., L]")
    dev, shape = nll.device, nll.shape
    lead, L = shape[:-1], shape[-1]
    a, lda = _scores(nll, shape, dev, "nll")
    o, ldo = _scores(old_nll, shape, dev, "old_nll")
    r, ldr = (None, 0) if ref_nll is None else _scores(ref_nll, shape, dev, "ref_nll")
    if isinstance(advantages, torch.Tensor) and advantages.dim() == nll.dim():
        v, ldv = _scores(advantages, shape, dev, "advantages")
    else:
        if not isinstance(advantages, torch.Tensor) or advantages.dtype != torch.float32 or advantages.device != dev or \
                advantages.shape != lead:
            raise ValueError(f"advantages must be a float32 tensor {list(lead)} or {list(shape)} on {dev}")
        v, ldv = advantages.contiguous(), 0
    n = _ints(lengths, lead, dev, "lengths")
    S = lead.numel()
    g = _loss_grad(grad, red, shape, dev)
    loss = _like(nll) if red == NONE else torch.empty((), dtype=torch.float32, device=dev)
    stats = torch.empty(2, dtype=torch.float32, device=dev)
    dnll = None if g is None else _like(nll)
    ws, nbytes = _status_or(workspace, policy_loss_workspace_size(S, L), dev)
    _run(dev, "ctcpb_policy_loss", a.data_ptr(), lda, o.data_ptr(), ldo, _p(r), ldr, v.data_ptr(), ldv, _p(n), S, L, clip_low,
         clip_high, kl_weight, red, _p(g), loss.data_ptr(), stats.data_ptr(), _p(dnll), _p(ws), nbytes)
    return (loss, stats) if g is None else (loss, stats, dnll)


def preference_loss_workspace_size(B: int, N: int, L: int) -> int:
    return _size("ctcpb_preference_loss_workspace_size", B, N, L)


def preference_loss(nll: torch.Tensor, chosen: torch.Tensor, rejected: torch.Tensor, *,
                    lengths: Optional[torch.Tensor] = None, ref_nll: Optional[torch.Tensor] = None, beta: float = 0.1,
                    margin: float = 0.0, label_smoothing: float = 0.0, average: bool = False, reduction: str = "mean",
                    grad: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """The preference loss of a pair of hypotheses of each N-best list: ``nll``
    [B, N, L] as in ``policy_loss``, ``chosen`` and ``rejected`` int32 [B] index the
    list (negative: the list takes no part), ``lengths`` int32 [B, N].  The
    log-ratios to ``ref_nll`` (0 without) are sums over tokens, or means with
    ``average``.  Returns (loss, margins [B]), the loss a scalar or [B] (reduction
    "none"); with ``grad`` (float32, a scalar or [B]) also dnll [B, N, L].
    ``D.read_status(workspace)`` holds ``DEV_TARGET`` if an index was N or more
    (such a list is ignored)."""
    red = _reduction(reduction)
    if not isinstance(nll, torch.Tensor) or not nll.is_cuda or nll.dim() != 3:
        raise ValueError("nll must be a CUDA float32 tensor [B, N, L]")
    dev, shape = nll.device, nll.shape
    B, N, L = shape
    a, lda = _scores(nll, shape, dev, "nll")
    r, ldr = (None, 0) if ref_nll is None else _scores(ref_nll, shape, dev, "ref_nll")
    if chosen is None or rejected is None:
        raise ValueError("chosen and rejected must be int32 tensors [B]")
    c, j = _ints(chosen, (B,), dev, "chosen"), _ints(rejected, (B,), dev, "rejected")
    n = _ints(lengths, (B, N), dev, "lengths")
    g = _loss_grad(grad, red, (B,), dev)
    loss = torch.empty((B,) if red == NONE else (), dtype=torch.float32, device=dev)
    margins = torch.empty((B,), dtype=torch.float32, device=dev)
    dnll = None if g is None else _like(nll)
    ws, nbytes = _status_or(workspace, preference_loss_workspace_size(B, N, L), dev)
    _run(dev, "ctcpb_preference_loss", a.data_ptr(), lda, _p(r), ldr, c.data_ptr(), j.data_ptr(), _p(n), B, N, L, beta, margin,
         label_smoothing, int(bool(average)), red, _p(g), loss.data_ptr(), margins.data_ptr(), _p(dnll), _p(ws), nbytes)
    return (loss, margins) if g is None else (loss, margins, dnll)
