"""Operators over vocabulary rows: top logits, one step of beam search, distillation from top logits.

Argument marshalling only, as in binding.py: every computation runs in the HIP library, asynchronous on the
current stream.  Logits are CUDA tensors [B, R, V] or [N, V], float32 or bfloat16, whose last dimension is
contiguous; slices of larger tensors and padded vocabularies are taken as they are.  The formulas, limits and
special cases are those of include/domino_head.h.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from .binding import DOMINO_BF16, DOMINO_F32, _check, _ptr, _stream_handle, load_library

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
        lib.domino_distill_workspace_size.argtypes = [LG, ctypes.POINTER(SZ)]
        lib.domino_distill.argtypes = [LG, I32, P, P, P, F32, P, P, SZ, P, P, P, LG, P]
        lib.domino_distill_backward.argtypes = [LG, I32, P, P, P, F32, P, LG, P]
        _declared = lib
    return lib


def _logits(name: str, t) -> Logits:
    if not isinstance(t, torch.Tensor) or t.dtype not in _DTYPES or t.dim() not in (2, 3) or not t.is_cuda or \
            (t.stride(-1) != 1 and t.shape[-1] != 1):
        raise ValueError("%s: expected a CUDA float32 or bfloat16 tensor [B, R, V] or [N, V] whose last dimension is "
                         "contiguous, got %s" % (name, _said(t)))
    if t.device.index != torch.cuda.current_device():
        raise ValueError("%s is on %s, the current device is cuda:%d" % (name, t.device, torch.cuda.current_device()))
    if t.dim() == 2:
        return Logits(t.data_ptr(), t.stride(0), t.shape[1], t.shape[0], 1, t.shape[1], _DTYPES[t.dtype])
    return Logits(t.data_ptr(), t.stride(0), t.stride(1), t.shape[0], t.shape[1], t.shape[2], _DTYPES[t.dtype])


def _said(t) -> str:
    return "%s %s on %s" % (t.dtype, tuple(t.shape), t.device) if isinstance(t, torch.Tensor) else type(t).__name__


def _need(name: str, t, shape, dtype, device):
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.shape != shape or t.device != device or \
            not t.is_contiguous():
        raise ValueError("%s: expected a contiguous %s tensor on %s of shape %s, got %s" %
                         (name, dtype, device, tuple(shape), _said(t)))


def _outputs(out: Optional[dict], wanted: dict, device) -> dict:
    """The output tensors by name: those of `out`, checked, and new ones for the rest."""
    out = {} if out is None else dict(out)
    for name in out:
        if name not in wanted:
            raise ValueError("out: unknown entry %r (expected %s)" % (name, ", ".join(wanted)))
    for name, (shape, dtype) in wanted.items():
        t = out.get(name)
        if t is None:
            out[name] = torch.empty(shape, dtype=dtype, device=device)
        else:
            _need("out[%r]" % name, t, shape, dtype, device)
    return out


def _workspace(given: Optional[torch.Tensor], size_fn, *args) -> torch.Tensor:
    n = ctypes.c_size_t()
    _check(size_fn(*args, ctypes.byref(n)))
    if given is None:
        return torch.empty(max(n.value, 16), dtype=torch.uint8, device="cuda")
    if not isinstance(given, torch.Tensor) or given.dtype != torch.uint8 or not given.is_cuda or \
            not given.is_contiguous():
        raise ValueError("workspace: expected a contiguous CUDA uint8 tensor, got %s" % _said(given))
    return given


def _size_of(fn, lg: Logits, *args) -> int:
    n = ctypes.c_size_t()
    _check(fn(ctypes.byref(lg), *args, ctypes.byref(n)))
    return int(n.value)


def _shape_only(B: int, R: int, V: int, dtype: torch.dtype) -> Logits:
    if dtype not in _DTYPES:
        raise ValueError("dtype %s is neither float32 nor bfloat16" % dtype)
    return Logits(None, 0, 0, B, R, V, _DTYPES[dtype])


def top_logits_workspace_size(B: int, R: int, V: int, k: int, dtype: torch.dtype = torch.float32) -> int:
    """Bytes of device workspace `top_logits` needs (host only)."""
    return _size_of(_lib().domino_top_logits_workspace_size, _shape_only(B, R, V, dtype), k)


def beam_step_workspace_size(B: int, W: int, V: int, n_out: int, dtype: torch.dtype = torch.float32) -> int:
    """Bytes of device workspace `beam_step` needs (host only)."""
    return _size_of(_lib().domino_beam_step_workspace_size, _shape_only(B, W, V, dtype), n_out)


def distill_workspace_size(B: int, R: int, V: int, dtype: torch.dtype = torch.float32) -> int:
    """Bytes of device workspace `distill` needs (host only)."""
    return _size_of(_lib().domino_distill_workspace_size, _shape_only(B, R, V, dtype))


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
    out = _outputs(out, {"ids": (lead + (k,), torch.int32), "values": (lead + (k,), torch.float32),
                         "lse": (lead, torch.float32)}, dev)
    if n_rows is not None:
        _need("n_rows", n_rows, (lg.B,), torch.int32, dev)
    ws = _workspace(workspace, lib.domino_top_logits_workspace_size, ctypes.byref(lg), k)
    _check(lib.domino_top_logits(ctypes.byref(lg), k, temperature, _ptr(n_rows), _ptr(ws), ws.numel(),
                                 _ptr(out["ids"]), _ptr(out["values"]), _ptr(out["lse"]), _stream_handle()))
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
    _need("scores", scores, (B, W), torch.float32, dev)
    bm = Beam(n_out=M, eos=eos, scores=scores.data_ptr())
    wanted = {"scores": ((B, M), torch.float32), "parent": ((B, M), torch.int32), "token": ((B, M), torch.int32)}
    if eos >= 0:
        wanted["finished"] = ((B, M), torch.bool)
    if finished is not None:
        _need("finished", finished, (B, W), torch.bool, dev)
        bm.finished = finished.data_ptr()
    if state is not None:
        if not isinstance(state, torch.Tensor) or state.dim() < 2:
            raise ValueError("state must be [B, W, ...]")
        _need("state", state, (B, W) + state.shape[2:], state.dtype, dev)
        bm.state, bm.state_bytes = state.data_ptr(), state.shape[2:].numel() * state.element_size()
        wanted["state"] = ((B, M) + state.shape[2:], state.dtype)
    if history is not None:
        if not isinstance(history, torch.Tensor) or history.dim() != 3:
            raise ValueError("history must be [B, W, T]")
        _need("history", history, (B, W, history.shape[2]), torch.int32, dev)
        bm.history, bm.T, bm.step = history.data_ptr(), history.shape[2], step
        wanted["history"] = ((B, M, history.shape[2]), torch.int32)
    out = _outputs(out, wanted, dev)
    for name, given in (("scores", scores), ("finished", finished), ("state", state), ("history", history)):
        if given is not None and name in out:
            if B and out[name].data_ptr() == given.data_ptr():
                raise ValueError("out[%r] is the input" % name)
    bm.out_scores, bm.out_parent, bm.out_token = (out["scores"].data_ptr(), out["parent"].data_ptr(),
                                                  out["token"].data_ptr())
    bm.out_finished = out["finished"].data_ptr() if eos >= 0 else None
    bm.out_state = out["state"].data_ptr() if state is not None else None
    bm.out_history = out["history"].data_ptr() if history is not None else None
    ws = _workspace(workspace, lib.domino_beam_step_workspace_size, ctypes.byref(lg), M)
    _check(lib.domino_beam_step(ctypes.byref(lg), ctypes.byref(bm), _ptr(ws), ws.numel(), _stream_handle()))
    return out


def distill(logits: torch.Tensor, ids: torch.Tensor, values: torch.Tensor, teacher_lse: Optional[torch.Tensor] = None,
            temperature: float = 1.0, n_rows: Optional[torch.Tensor] = None, grad_loss: Optional[torch.Tensor] = None,
            workspace: Optional[torch.Tensor] = None, out: Optional[dict] = None) -> dict:
    """Loss of the student's rows against a teacher's top logits, and with `grad_loss` its gradient.

    logits [B, R, V] (or [N, V]) of the student; ids int32 and values float32 [B, R, k] of the teacher
    (`top_logits`); teacher_lse [B, R] float32 at the same temperature: the mass of all other ids is then one
    more event, without it the teacher is its entries alone.  n_rows [B] int32: rows r >= n_rows[b] are left
    out (loss and gradient 0).

    Returns loss [B, R] float32 (temperature^2 times the divergence) and stats [B, R, 4 + k] float32 for
    `distill_backward`; with grad_loss [B, R] float32 also grad = grad_loss * dloss/dlogits, of the logits'
    shape and type.  ``out`` may supply these tensors (grad may be the logits themselves, or any tensor of
    their shape and type with a contiguous last dimension), ``workspace`` (uint8) the scratch.
    """
    lib = _lib()
    lg = _logits("logits", logits)
    dev, lead = logits.device, logits.shape[:-1]
    k = _teacher_ids(ids, lead, dev)
    _need("values", values, ids.shape, torch.float32, dev)
    if teacher_lse is not None:
        _need("teacher_lse", teacher_lse, lead, torch.float32, dev)
    if n_rows is not None:
        _need("n_rows", n_rows, (lg.B,), torch.int32, dev)
    out = {} if out is None else dict(out)
    grad = None
    if grad_loss is not None:
        _need("grad_loss", grad_loss, lead, torch.float32, dev)
        grad = out.pop("grad", None)
        if grad is None:
            grad = torch.empty(logits.shape, dtype=logits.dtype, device=dev)
    gd = None if grad is None else _grad("out['grad']", grad, logits)
    out = _outputs(out, {"loss": (lead, torch.float32), "stats": (lead + (STAT_HEAD + k,), torch.float32)}, dev)
    ws = _workspace(workspace, lib.domino_distill_workspace_size, ctypes.byref(lg))
    _check(lib.domino_distill(ctypes.byref(lg), k, _ptr(ids), _ptr(values), _ptr(teacher_lse), temperature,
                              _ptr(n_rows), _ptr(ws), ws.numel(), _ptr(out["loss"]), _ptr(out["stats"]),
                              _ptr(grad_loss), None if gd is None else ctypes.byref(gd), _stream_handle()))
    if grad is not None:
        out["grad"] = grad
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
    _need("stats", stats, lead + (STAT_HEAD + k,), torch.float32, dev)
    _need("grad_loss", grad_loss, lead, torch.float32, dev)
    if n_rows is not None:
        _need("n_rows", n_rows, (lg.B,), torch.int32, dev)
    if out is None:
        out = torch.empty(logits.shape, dtype=logits.dtype, device=dev)
    gd = _grad("out", out, logits)
    _check(lib.domino_distill_backward(ctypes.byref(lg), k, _ptr(ids), _ptr(stats), _ptr(grad_loss), temperature,
                                       _ptr(n_rows), ctypes.byref(gd), _stream_handle()))
    return out


def _teacher_ids(ids, lead, device) -> int:
    if not isinstance(ids, torch.Tensor) or ids.dim() != len(lead) + 1:
        raise ValueError("ids: expected a tensor of shape %s, got %s" % (tuple(lead) + ("k",), _said(ids)))
    _need("ids", ids, lead + ids.shape[-1:], torch.int32, device)
    return ids.shape[-1]


def _grad(name: str, grad, logits: torch.Tensor) -> Logits:
    gd = _logits(name, grad)
    if grad.shape != logits.shape or grad.dtype != logits.dtype or grad.device != logits.device:
        raise ValueError("%s: expected a %s tensor on %s of shape %s, got %s" %
                         (name, logits.dtype, logits.device, tuple(logits.shape), _said(grad)))
    return gd
