"""Layers over rows: embedding, linear, and their gradients.

Argument marshalling only, as in rows.py: every computation runs in the HIP library, asynchronous on the current
stream.  Operands are CUDA tensors [B, R, V] or [N, V], float32 or bfloat16 each for itself, whose last dimension is
contiguous; slices of larger tensors are taken as they are.  The formulas, limits and special cases are those of
include/domino_head.h.  No graph is recorded: the gradients are what the backward calls return.
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional

import torch

from .binding import _check, load_library
from .rows import _DTYPES, _LOGITS, _known, _logits, _said, _scratch, _shape_only, _size_of, _stream

ACTIVATIONS = {None: 0, "silu": 1, "gelu": 2, "relu": 3}
_LINEAR_OUT, _LINEAR_GRADS = {"y", "pre"}, ("x", "weight", "bias")

_declared = None


def _lib():
    global _declared
    lib = load_library()
    if _declared is not lib:
        P, I32, F64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_double, ctypes.c_size_t
        lib.domino_embed.argtypes = [P, P, F64, P, P]
        lib.domino_embed_backward_workspace_size.argtypes = [P, ctypes.POINTER(SZ)]
        lib.domino_embed_backward.argtypes = [P, P, F64, I32, P, SZ, P, P]
        lib.domino_linear_workspace_size.argtypes = [P, P, I32, ctypes.POINTER(SZ)]
        lib.domino_linear.argtypes = [P, P, P, I32, P, P, SZ, P, P, P]
        lib.domino_linear_backward_workspace_size.argtypes = [P, P, P, I32, I32, I32, I32, ctypes.POINTER(SZ)]
        lib.domino_linear_backward.argtypes = [P, P, P, P, I32, I32, P, SZ, P, P, P, P]
        _declared = lib
    return lib


def _matrix(name: str, t):
    """(the packed domino_rows, rows, columns, device index) of one matrix."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError("%s: expected a tensor of two dimensions, got %s" % (name, _said(t)))
    gpu = _logits(name, t)[-1]
    n, d = t.shape
    return _LOGITS(t.data_ptr(), 0, t.stride(0), 1, n, d, _DTYPES[t.dtype]), n, d, gpu


def _ids(ids, lead, gpu: int) -> int:
    if not isinstance(ids, torch.Tensor) or ids.dtype is not torch.int32 or ids.get_device() != gpu or \
            not ids.is_contiguous() or (lead is not None and ids.shape != lead):
        raise ValueError("ids: expected a contiguous int32 tensor on cuda:%d%s, got %s" %
                         (gpu, "" if lead is None else " of shape %s" % (tuple(lead),), _said(ids)))
    return ids.data_ptr()


def _no_graph(what: str, *tensors):
    """Refuses inputs whose gradients a caller may expect autograd to know."""
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors):
        raise ValueError("an input requires a gradient, of which %s records nothing: detach it (or use no_grad) and "
                         "call %s_backward" % (what, what))


def embed(table: torch.Tensor, ids: torch.Tensor, scale: float = 1.0, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """scale * table[ids]: a row of the table for each token, zeros for ids outside it.

    table [V, d]; ids [N] or [B, R] int32.  Returns [..., d] of the table's type; ``out`` may supply it, as float32 or
    bfloat16.
    """
    lib = _declared or _lib()
    tb, _, d, gpu = _matrix("table", table)
    _no_graph("embed", table)
    at = _ids(ids, None, gpu)
    if ids.dim() not in (1, 2):
        raise ValueError("ids must be [N] or [B, R], got %s" % _said(ids))
    if out is None:
        out = torch.empty(tuple(ids.shape) + (d,), dtype=table.dtype, device="cuda")
    elif not isinstance(out, torch.Tensor) or out.shape != ids.shape + (d,):
        raise ValueError("out: expected a tensor of shape %s, got %s" % (tuple(ids.shape) + (d,), _said(out)))
    if ids.numel():
        _check(lib.domino_embed(tb, at, scale, _logits("out", out)[0], _stream(gpu)))
    return out


@functools.lru_cache(maxsize=1024)
def embed_backward_workspace_size(B: int, R: int, d: int) -> int:
    """Bytes of device workspace `embed_backward` needs for [B, R, d] gradients (host only)."""
    return _size_of(_lib().domino_embed_backward_workspace_size, _shape_only(B, R, d, torch.float32))


def embed_backward(grad: torch.Tensor, ids: torch.Tensor, V: int, scale: float = 1.0, accumulate: bool = False,
                   dtype: Optional[torch.dtype] = None, workspace: Optional[torch.Tensor] = None,
                   out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The gradient [V, d] of `embed`'s table: row v is scale times the sum of grad over the places where ids is v.

    grad [N, d] or [B, R, d]; ids int32 of the shape before it; ids outside [0, V) are passed over.  The gradient is
    of `dtype` (default: grad's), or ``out``, float32 or bfloat16; with `accumulate` the sums are added to ``out``,
    whose other rows stay as they are.  The same inputs give the same bits.  ``workspace`` (uint8) may supply the scratch.
    """
    lib = _declared or _lib()
    gd, B, R, d, gpu = _logits("grad", grad)
    at = _ids(ids, grad.shape[:-1], gpu)
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs the tensor to add to, as out")
        out = torch.empty((V, d), dtype=dtype or grad.dtype, device="cuda")
    elif not isinstance(out, torch.Tensor) or out.shape != (V, d) or (dtype is not None and out.dtype is not dtype):
        raise ValueError("out: expected a tensor of shape %s%s, got %s" %
                         ((V, d), "" if dtype is None else " and type %s" % dtype, _said(out)))
    if not B * R:
        gd, at = _LOGITS(0, 0, 0, 0, 1, d, _DTYPES[grad.dtype]), None
        B = 0
    _ws, ws, ws_bytes = _scratch(workspace, embed_backward_workspace_size(B, R if B else 1, d), gpu)
    _check(lib.domino_embed_backward(gd, at, scale, bool(accumulate), ws, ws_bytes, _matrix("out", out)[0],
                                     _stream(gpu)))
    return out


def _act(activation) -> int:
    if activation not in ACTIVATIONS:
        raise ValueError("activation %r is none of %s" % (activation, list(ACTIVATIONS)))
    return ACTIVATIONS[activation]


def _rows_like(name: str, t, shape) -> bytes:
    packed = _logits(name, t)[0]
    if t.shape != shape:
        raise ValueError("%s: expected a tensor of shape %s, got %s" % (name, tuple(shape), _said(t)))
    return packed


def _vector(name: str, t, n: int, gpu: int) -> bytes:
    dtype = _DTYPES.get(t.dtype) if isinstance(t, torch.Tensor) else None
    if dtype is None or t.shape != (n,) or t.get_device() != gpu or not t.is_contiguous():
        raise ValueError("%s: expected a contiguous float32 or bfloat16 tensor on cuda:%d of shape %s, got %s" %
                         (name, gpu, (n,), _said(t)))
    return _LOGITS(t.data_ptr(), 0, 0, 1, 1, n, dtype)


@functools.lru_cache(maxsize=1024)
def linear_workspace_size(B: int, R: int, K: int, N: int, activation: Optional[str] = None,
                          dtypes: tuple = (torch.float32, torch.float32)) -> int:
    """Bytes of device workspace `linear` needs for x [B, R, K] and weight [N, K] of these types (host only)."""
    w = _shape_only(1, N, K, dtypes[1])
    return _size_of(_lib().domino_linear_workspace_size, _shape_only(B, R, K, dtypes[0]), ctypes.byref(w),
                    _act(activation))


@functools.lru_cache(maxsize=1024)
def linear_backward_workspace_size(B: int, R: int, K: int, N: int, activation: Optional[str] = None,
                                   want: tuple = ("x", "weight"),
                                   dtypes: tuple = (torch.float32, torch.float32, torch.float32)) -> int:
    """Bytes of device workspace `linear_backward` needs for grad [B, R, N], x [B, R, K] and weight [N, K] of these
    types (host only)."""
    x, w = _shape_only(B, R, K, dtypes[1]), _shape_only(1, N, K, dtypes[2])
    return _size_of(_lib().domino_linear_backward_workspace_size, _shape_only(B, R, N, dtypes[0]), ctypes.byref(x),
                    ctypes.byref(w), _act(activation), *(name in want for name in _LINEAR_GRADS))


def linear(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
           activation: Optional[str] = None, residual: Optional[torch.Tensor] = None, want_pre: bool = False,
           dtype: Optional[torch.dtype] = None, workspace: Optional[torch.Tensor] = None,
           out: Optional[dict] = None) -> dict:
    """y = act(x weight^T + bias) + residual.

    x [B, R, K] or [N, K]; weight [n, K]; bias [n]; residual [..., n]; activation None, "silu", "gelu" (with the normal
    distribution's function) or "relu".  Returns y [..., n] of `dtype` (default: the residual's type, else x's) and
    with want_pre pre [..., n] float32, x weight^T + bias, which `linear_backward` takes where there is an activation.
    ``out`` may supply these tensors, each float32 or bfloat16 (y may be the residual), ``workspace`` (uint8) the
    scratch.
    """
    lib = _declared or _lib()
    xd, B, R, K, gpu = _logits("x", x)
    wd, n, _, _ = _matrix("weight", weight)
    _no_graph("linear", x, weight, bias, residual)
    act = _act(activation)
    shape = x.shape[:-1] + (n,)
    out = _known(out, _LINEAR_OUT)
    if out.get("y") is None:
        out["y"] = torch.empty(shape, dtype=dtype or (x if residual is None else residual).dtype, device="cuda")
    elif dtype is not None and out["y"].dtype is not dtype:
        raise ValueError("out['y']: expected type %s, got %s" % (dtype, _said(out["y"])))
    if want_pre and out.get("pre") is None:
        out["pre"] = torch.empty(shape, dtype=torch.float32, device="cuda")
    yd = _rows_like("out['y']", out["y"], shape)
    pd = None if out.get("pre") is None else _rows_like("out['pre']", out["pre"], shape)
    rd = None if residual is None else _rows_like("residual", residual, shape)
    bd = None if bias is None else _vector("bias", bias, n, gpu)
    if B * R:
        _ws, ws, ws_bytes = _scratch(workspace, linear_workspace_size(B, R, K, n, activation, (x.dtype, weight.dtype)),
                                     gpu)
        _check(lib.domino_linear(xd, wd, bd, act, rd, ws, ws_bytes, yd, pd, _stream(gpu)))
    return out


def linear_backward(grad: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, pre: Optional[torch.Tensor] = None,
                    activation: Optional[str] = None, want: tuple = ("x", "weight"), accumulate: bool = False,
                    workspace: Optional[torch.Tensor] = None, out: Optional[dict] = None) -> dict:
    """The gradients of `linear`'s x, weight and bias (those that `want` names) from grad [..., n], that of its y.

    x and weight as in the forward call; pre [..., n] from it, where there is an activation.  Returns x [..., K] and
    weight [n, K], of the types of these, and bias [n] float32; ``out`` may supply tensors for them, each float32 or
    bfloat16.  With `accumulate` the gradients of weight and bias are added to the tensors that ``out`` has for them.
    ``workspace`` (uint8) may supply the scratch.  The residual's gradient is grad itself.
    """
    lib = _declared or _lib()
    gd, B, R, n, gpu = _logits("grad", grad)
    xd, _, _, K, _ = _logits("x", x)
    wd, wn, _, _ = _matrix("weight", weight)
    if x.shape[:-1] != grad.shape[:-1] or wn != n or weight.shape[1] != K:
        raise ValueError("grad %s, x %s and weight %s do not belong together" %
                         (tuple(grad.shape), tuple(x.shape), tuple(weight.shape)))
    act = _act(activation)
    want = tuple(name for name in _LINEAR_GRADS if name in want) if set(want) <= set(_LINEAR_GRADS) else ()
    if not want:
        raise ValueError("want: some of %s" % (_LINEAR_GRADS,))
    out = _known(out, set(want))
    if accumulate and any(out.get(name) is None for name in want if name != "x"):
        raise ValueError("accumulate needs the tensors to add to, as out")
    pd = None if pre is None else _rows_like("pre", pre, grad.shape)
    dx = dw = db = None
    if "x" in want:
        if out.get("x") is None:
            out["x"] = torch.empty(x.shape, dtype=x.dtype, device="cuda")
        dx = _rows_like("out['x']", out["x"], x.shape)
    if "weight" in want:
        if out.get("weight") is None:
            out["weight"] = torch.empty((n, K), dtype=weight.dtype, device="cuda")
        dw, dn, dk, _ = _matrix("out['weight']", out["weight"])
        if (dn, dk) != (n, K):
            raise ValueError("out['weight']: expected a tensor of shape %s, got %s" % ((n, K), _said(out["weight"])))
    if "bias" in want:
        if out.get("bias") is None:
            out["bias"] = torch.empty(n, dtype=torch.float32, device="cuda")
        db = _vector("out['bias']", out["bias"], n, gpu)
    if not B * R:  # (a tensor without rows may have R = 0)
        none = [_LOGITS(0, 0, 0, 0, 1, v, 0) for v in (n, K)]
        gd, xd, dx, pd, B, R = none[0], none[1], None if dx is None else none[1], None if pd is None else none[0], 0, 1
    need = linear_backward_workspace_size(B, R, K, n, activation, want, (grad.dtype, x.dtype, weight.dtype))
    _ws, ws, ws_bytes = _scratch(workspace, need, gpu)
    _check(lib.domino_linear_backward(gd, xd, wd, pd, act, bool(accumulate), ws, ws_bytes, dx, dw, db, _stream(gpu)))
    return out
