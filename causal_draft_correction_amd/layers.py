"""Layers over rows: embedding, and its gradient.

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
from .rows import _DTYPES, _LOGITS, _logits, _said, _scratch, _shape_only, _size_of, _stream

_declared = None


def _lib():
    global _declared
    lib = load_library()
    if _declared is not lib:
        P, I32, F64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_double, ctypes.c_size_t
        lib.domino_embed.argtypes = [P, P, F64, P, P]
        lib.domino_embed_backward_workspace_size.argtypes = [P, ctypes.POINTER(SZ)]
        lib.domino_embed_backward.argtypes = [P, P, F64, I32, P, SZ, P, P]
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
