"""Operators over vocabulary rows: top logits, one step of beam search, distillation from top logits.

Argument marshalling only, as in binding.py: every computation runs in the HIP library, asynchronous on the
current stream.  Logits are CUDA tensors [B, R, V] or [N, V], float32 or bfloat16, whose last dimension is
contiguous; slices of larger tensors and padded vocabularies are taken as they are.  The formulas, limits and
special cases are those of include/domino_head.h.
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional

import torch

from .binding import DOMINO_BF16, DOMINO_F32, _check, load_library

STAT_HEAD = 4  # floats of a row's statistics before those of its ids
_DTYPES = {torch.float32: DOMINO_F32, torch.bfloat16: DOMINO_BF16}


class Logits(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("batch_stride", ctypes.c_int64), ("row_stride", ctypes.c_int64),
                ("B", ctypes.c_int32), ("R", ctypes.c_int32), ("V", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class Beam(ctypes.Structure):
    _fields_ = [("n_out", ctypes.c_int32), ("eos", ctypes.c_int32), ("T", ctypes.c_int32), ("step", ctypes.c_int32),
                ("state_bytes", ctypes.c_int64), ("scores", ctypes.c_void_p), ("finished", ctypes.c_void_p),
                ("state", ctypes.c_void_p), ("history", ctypes.c_void_p), ("out_scores", ctypes.c_void_p),
                ("out_parent", ctypes.c_void_p), ("out_token", ctypes.c_void_p), ("out_finished", ctypes.c_void_p),
                ("out_state", ctypes.c_void_p), ("out_history", ctypes.c_void_p)]


_declared = None


def _lib():
    global _declared
    lib = load_library()
    if _declared is not lib:
        P, I32, F32, SZ, LG = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t,
                               ctypes.POINTER(Logits))
        lib.domino_top_logits_workspace_size.argtypes = [LG, I32, ctypes.POINTER(SZ)]
        lib.domino_top_logits.argtypes = [LG, I32, F32, P, P, SZ, P, P, P, P]
        lib.domino_beam_step_workspace_size.argtypes = [LG, I32, ctypes.POINTER(SZ)]
        lib.domino_beam_step.argtypes = [LG, ctypes.POINTER(Beam), P, SZ, P]
        lib.domino_distill_workspace_size.argtypes = [LG, I32, ctypes.POINTER(SZ)]
        lib.domino_distill.argtypes = [LG, I32, P, P, P, F32, P, P, SZ, P, P, P, LG, P]
        lib.domino_distill_backward.argtypes = [LG, I32, P, P, P, F32, P, LG, P]
        _declared = lib
    return lib


def _logits(name: str, t) -> Logits:
    dtype = _DTYPES.get(t.dtype) if isinstance(t, torch.Tensor) else None
    shape = t.shape if dtype is not None else ()
    if len(shape) not in (2, 3) or not t.is_cuda or (t.stride(-1) != 1 and shape[-1] != 1):
        raise ValueError("%s: expected a CUDA float32 or bfloat16 tensor [B, R, V] or [N, V] whose last dimension is "
                         "contiguous, got %s" % (name, _said(t)))
    if t.get_device() != torch.cuda.current_device():
        raise ValueError("%s is on %s, the current device is cuda:%d" % (name, t.device, torch.cuda.current_device()))
    if len(shape) == 2:
        return Logits(t.data_ptr(), t.stride(0), shape[1], shape[0], 1, shape[1], dtype)
    return Logits(t.data_ptr(), t.stride(0), t.stride(1), shape[0], shape[1], shape[2], dtype)


def _said(t) -> str:
    return "%s %s on %s" % (t.dtype, tuple(t.shape), t.device) if isinstance(t, torch.Tensor) else type(t).__name__


def _need(name: str, t, shape, dtype, device) -> int:
    """The tensor's address, if it is a contiguous one of this shape and type."""
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.shape != shape or t.device != device or \
            not t.is_contiguous():
        raise ValueError("%s: expected a contiguous %s tensor on %s of shape %s, got %s" %
                         (name, dtype, device, tuple(shape), _said(t)))
    return t.data_ptr()


def _maybe(name: str, t, shape, dtype, device):
    return None if t is None else _need(name, t, shape, dtype, device)


def _output(out: dict, name: str, shape, dtype, device) -> int:
    """The address of output `name`: the caller's tensor, checked, or a new one."""
    t = out.get(name)
    if t is None:
        t = out[name] = torch.empty(shape, dtype=dtype, device=device)
        return t.data_ptr()
    return _need("out[%r]" % name, t, shape, dtype, device)


def _known(out: Optional[dict], names) -> dict:
    out = {} if out is None else dict(out)
    for name in out:
        if name not in names:
            raise ValueError("out: unknown entry %r (expected %s)" % (name, ", ".join(names)))
    return out


def _scratch(given: Optional[torch.Tensor], need: int, device) -> torch.Tensor:
    if given is None:
        return torch.empty(need, dtype=torch.uint8, device=device)
    if not isinstance(given, torch.Tensor) or given.dtype != torch.uint8 or given.device != device or \
            not given.is_contiguous():
        raise ValueError("workspace: expected a contiguous uint8 tensor on %s, got %s" % (device, _said(given)))
    return given


def _stream(logits: torch.Tensor) -> int:
    """The current stream's handle (torch.cuda.current_stream() builds a Stream object around it each time)."""
    return torch._C._cuda_getCurrentRawStream(logits.get_device())


def _size_of(fn, lg: Logits, *args) -> int:
    n = ctypes.c_size_t()
    _check(fn(ctypes.byref(lg), *args, ctypes.byref(n)))
    return int(n.value)


def _shape_only(B: int, R: int, V: int, dtype: torch.dtype) -> Logits:
    if dtype not in _DTYPES:
        raise ValueError("dtype %s is neither float32 nor bfloat16" % dtype)
    return Logits(None, 0, 0, B, R, V, _DTYPES[dtype])


@functools.lru_cache(maxsize=1024)
def top_logits_workspace_size(B: int, R: int, V: int, k: int, dtype: torch.dtype = torch.float32) -> int:
    """Bytes of device workspace `top_logits` needs (host only)."""
    return _size_of(_lib().domino_top_logits_workspace_size, _shape_only(B, R, V, dtype), k)


@functools.lru_cache(maxsize=1024)
def beam_step_workspace_size(B: int, W: int, V: int, n_out: int, dtype: torch.dtype = torch.float32) -> int:
    """Bytes of device workspace `beam_step` needs (host only)."""
    return _size_of(_lib().domino_beam_step_workspace_size, _shape_only(B, W, V, dtype), n_out)


@functools.lru_cache(maxsize=1024)
def distill_workspace_size(B: int, R: int, V: int, k: int, dtype: torch.dtype = torch.float32) -> int:
    """Bytes of device workspace `distill` needs (host only)."""
    return _size_of(_lib().domino_distill_workspace_size, _shape_only(B, R, V, dtype), k)


def top_logits(logits: torch.Tensor, k: int, temperature: float = 1.0, n_rows: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None, out: Optional[dict] = None) -> dict:
    """The k largest logits of every row, and the row's log-sum-exp at `temperature`.

    logits [B, R, V] (or [N, V]).  n_rows [B] int32: rows r >= n_rows[b] are left out.  Returns ids [B, R, k]
    int32 and values [B, R, k] float32, largest first with ties to the lowest id, and lse [B, R] float32 (-1,
    -inf and -inf in rows left out).  ``out`` may supply these tensors, ``workspace`` (uint8) the scratch.
    """
    lib = _lib()
    lg = _logits("logits", logits)
    dev, lead = logits.device, logits.shape[:-1]
    need = top_logits_workspace_size(lg.B, lg.R, lg.V, k, logits.dtype)
    out = _known(out, ("ids", "values", "lse"))
    ids = _output(out, "ids", lead + (k,), torch.int32, dev)
    values = _output(out, "values", lead + (k,), torch.float32, dev)
    lse = _output(out, "lse", lead, torch.float32, dev)
    rows = _maybe("n_rows", n_rows, (lg.B,), torch.int32, dev)
    ws = _scratch(workspace, need, dev)
    _check(lib.domino_top_logits(ctypes.byref(lg), k, temperature, rows, ws.data_ptr(), ws.numel(), ids, values, lse,
                                 _stream(logits)))
    return out


def beam_step(logits: torch.Tensor, scores: torch.Tensor, n_out: Optional[int] = None, eos: int = -1,
              finished: Optional[torch.Tensor] = None, state: Optional[torch.Tensor] = None,
              history: Optional[torch.Tensor] = None, step: int = 0, workspace: Optional[torch.Tensor] = None,
              out: Optional[dict] = None) -> dict:
    """One step of beam search: the n_out best continuations of each batch entry's beams.

    logits [B, W, V]; scores [B, W] float32 sums of log-probabilities (-inf: a dead beam, so a search starts
    from [0, -inf, ...]); finished [B, W] bool: beams that have ended (with `eos`); state [B, W, ...] any
    tensor of per-beam state, 4 bytes or a multiple a beam; history [B, W, T] int32, in which the new token
    takes place `step`.  n_out defaults to W.

    Returns scores [B, n_out] float32, parent and token [B, n_out] int32, finished [B, n_out] bool (with
    eos >= 0), state and history in the new order (where given).  ``out`` may supply these tensors,
    ``workspace`` (uint8) the scratch; outputs may not be the inputs.
    """
    lib = _lib()
    lg = _logits("logits", logits)
    if logits.dim() != 3:
        raise ValueError("logits must be [B, W, V]")
    dev, (B, W, V) = logits.device, logits.shape
    M = W if n_out is None else n_out
    need = beam_step_workspace_size(B, W, V, M, logits.dtype)
    out = _known(out, ("scores", "parent", "token") + (("finished",) if eos >= 0 else ()) +
                 (("state",) if state is not None else ()) + (("history",) if history is not None else ()))
    given = {"scores": _need("scores", scores, (B, W), torch.float32, dev),
             "finished": _maybe("finished", finished, (B, W), torch.bool, dev), "state": None, "history": None}
    state_bytes = T = 0
    o_finished = o_state = o_history = None
    o_scores = _output(out, "scores", (B, M), torch.float32, dev)
    o_parent = _output(out, "parent", (B, M), torch.int32, dev)
    o_token = _output(out, "token", (B, M), torch.int32, dev)
    if eos >= 0:
        o_finished = _output(out, "finished", (B, M), torch.bool, dev)
    if state is not None:
        if not isinstance(state, torch.Tensor) or state.dim() < 2:
            raise ValueError("state must be [B, W, ...]")
        one = state.shape[2:]
        given["state"] = _need("state", state, (B, W) + one, state.dtype, dev)
        o_state = _output(out, "state", (B, M) + one, state.dtype, dev)
        state_bytes = one.numel() * state.element_size()
    if history is not None:
        if not isinstance(history, torch.Tensor) or history.dim() != 3:
            raise ValueError("history must be [B, W, T]")
        T = history.shape[2]
        given["history"] = _need("history", history, (B, W, T), torch.int32, dev)
        o_history = _output(out, "history", (B, M, T), torch.int32, dev)
    if B and (o_scores == given["scores"] or (o_state and o_state == given["state"]) or
              (o_history and o_history == given["history"]) or (o_finished and o_finished == given["finished"])):
        raise ValueError("out: an output tensor is the input it is made from")
    bm = Beam(M, eos, T, step, state_bytes, given["scores"], given["finished"], given["state"], given["history"],
              o_scores, o_parent, o_token, o_finished, o_state, o_history)
    ws = _scratch(workspace, need, dev)
    _check(lib.domino_beam_step(ctypes.byref(lg), ctypes.byref(bm), ws.data_ptr(), ws.numel(), _stream(logits)))
    return out


def distill(logits: torch.Tensor, ids: torch.Tensor, values: torch.Tensor, teacher_lse: Optional[torch.Tensor] = None,
            temperature: float = 1.0, n_rows: Optional[torch.Tensor] = None, grad_loss: Optional[torch.Tensor] = None,
            workspace: Optional[torch.Tensor] = None, out: Optional[dict] = None) -> dict:
    """Loss of the student's rows against a teacher's top logits, and with `grad_loss` its gradient.

    logits [B, R, V] (or [N, V]) of the student; ids int32 and values float32 [B, R, k] of the teacher
    (`top_logits`); teacher_lse [B, R] float32 at the same temperature: the mass of all other ids is then one
    more event, without it the teacher is its entries alone.  n_rows [B] int32: rows r >= n_rows[b] are left
    out (loss and gradient 0).

    Returns loss [B, R] float32 (temperature^2 times the divergence).  Without grad_loss also stats
    [B, R, 4 + k] float32 for `distill_backward`; with grad_loss [B, R] float32 instead grad = grad_loss *
    dloss/dlogits, of the logits' shape and type.  ``out`` may supply these tensors (grad may be the logits
    themselves, or any tensor of their shape and type with a contiguous last dimension), ``workspace`` (uint8)
    the scratch.
    """
    lib = _lib()
    lg = _logits("logits", logits)
    dev, lead = logits.device, logits.shape[:-1]
    k = _teacher_ids(ids, lead, dev)
    need = distill_workspace_size(lg.B, lg.R, lg.V, k, logits.dtype)
    v_ptr = _need("values", values, ids.shape, torch.float32, dev)
    lse = _maybe("teacher_lse", teacher_lse, lead, torch.float32, dev)
    rows = _maybe("n_rows", n_rows, (lg.B,), torch.int32, dev)
    g_ptr = _maybe("grad_loss", grad_loss, lead, torch.float32, dev)
    stats = gd = None
    if grad_loss is None:
        out = _known(out, ("loss", "stats"))
        stats = _output(out, "stats", lead + (STAT_HEAD + k,), torch.float32, dev)
    else:
        out = _known(out, ("loss", "grad"))
        if out.get("grad") is None:
            out["grad"] = torch.empty(logits.shape, dtype=logits.dtype, device=dev)
        gd = ctypes.byref(_grad("out['grad']", out["grad"], logits))
    loss = _output(out, "loss", lead, torch.float32, dev)
    ws = _scratch(workspace, need, dev)
    _check(lib.domino_distill(ctypes.byref(lg), k, ids.data_ptr(), v_ptr, lse, temperature, rows, ws.data_ptr(),
                              ws.numel(), loss, stats, g_ptr, gd, _stream(logits)))
    return out


def distill_backward(logits: torch.Tensor, ids: torch.Tensor, stats: torch.Tensor, grad_loss: torch.Tensor,
                     temperature: float = 1.0, n_rows: Optional[torch.Tensor] = None,
                     out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """grad_loss * dloss/dlogits of an earlier `distill` call, from its logits, ids and stats.

    grad_loss [B, R] float32; temperature and n_rows as in that call.  ``out`` may be the logits themselves, or
    any tensor of their shape and type with a contiguous last dimension.
    """
    lib = _lib()
    lg = _logits("logits", logits)
    dev, lead = logits.device, logits.shape[:-1]
    k = _teacher_ids(ids, lead, dev)
    s_ptr = _need("stats", stats, lead + (STAT_HEAD + k,), torch.float32, dev)
    g_ptr = _need("grad_loss", grad_loss, lead, torch.float32, dev)
    rows = _maybe("n_rows", n_rows, (lg.B,), torch.int32, dev)
    if out is None:
        out = torch.empty(logits.shape, dtype=logits.dtype, device=dev)
    gd = _grad("out", out, logits)
    _check(lib.domino_distill_backward(ctypes.byref(lg), k, ids.data_ptr(), s_ptr, g_ptr, temperature, rows,
                                       ctypes.byref(gd), _stream(logits)))
    return out


def _teacher_ids(ids, lead, device) -> int:
    if not isinstance(ids, torch.Tensor) or ids.dim() != len(lead) + 1:
        raise ValueError("ids: expected a tensor of shape %s, got %s" % (tuple(lead) + ("k",), _said(ids)))
    _need("ids", ids, lead + ids.shape[-1:], torch.int32, device)
    return ids.shape[-1]


def _grad(name: str, grad, logits: torch.Tensor) -> Logits:
    gd = _logits(name, grad)
    if grad.shape != logits.shape or grad.dtype != logits.dtype:
        raise ValueError("%s: expected a %s tensor on %s of shape %s, got %s" %
                         (name, logits.dtype, logits.device, tuple(logits.shape), _said(grad)))
    return gd
