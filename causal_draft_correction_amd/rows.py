"""Operators over vocabulary rows: top logits, one step of beam search, distillation from top logits.

Argument marshalling only, as in binding.py: every computation runs in the HIP library, asynchronous on the
current stream.  Logits are CUDA tensors [B, R, V] or [N, V], float32 or bfloat16, whose last dimension is
contiguous; slices of larger tensors and padded vocabularies are taken as they are.  The formulas, limits and
special cases are those of include/domino_head.h.
"""
from __future__ import annotations

import ctypes
import functools
import struct
from typing import Optional

import torch

from .binding import DOMINO_BF16, DOMINO_F32, _check, load_library

STAT_HEAD = 4  # floats of a row's statistics before those of its ids
_TOP_OUT, _LOSS_ONLY, _LOSS_OUT, _GRAD_OUT = {"ids", "values", "lse"}, {"loss"}, {"loss", "stats"}, {"loss", "grad"}
_BEAM_OUT = {"scores", "parent", "token", "finished", "state", "history"}
_DTYPES = {torch.float32: DOMINO_F32, torch.bfloat16: DOMINO_BF16}


# domino_logits and domino_beam as bytes, which take less time to make than their ctypes forms below
_LOGITS = struct.Struct("=Qqqiiii").pack
_BEAM = struct.Struct("=iiiiq10Q").pack


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
        P, I32, F64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_double, ctypes.c_size_t
        lib.domino_top_logits_workspace_size.argtypes = [P, I32, ctypes.POINTER(SZ)]
        lib.domino_top_logits.argtypes = [P, I32, F64, P, P, SZ, P, P, P, P]
        lib.domino_beam_step_workspace_size.argtypes = [P, I32, ctypes.POINTER(SZ)]
        lib.domino_beam_step.argtypes = [P, P, P, SZ, P]
        lib.domino_distill_workspace_size.argtypes = [P, I32, ctypes.POINTER(SZ)]
        lib.domino_distill.argtypes = [P, I32, P, P, P, F64, P, P, SZ, P, P, P, P, P]
        lib.domino_distill_backward.argtypes = [P, I32, P, P, P, F64, P, P, P]
        _declared = lib
    return lib


def _said(t) -> str:
    return "%s %s on %s" % (t.dtype, tuple(t.shape), t.device) if isinstance(t, torch.Tensor) else type(t).__name__


def _logits(name: str, t):
    """(the packed domino_logits, B, R, V, device index) of a tensor of logits."""
    dtype = _DTYPES.get(t.dtype) if isinstance(t, torch.Tensor) else None
    shape = t.shape if dtype is not None else ()
    n = len(shape)
    if (n != 3 and n != 2) or not t.is_cuda:
        raise ValueError("%s: expected a CUDA float32 or bfloat16 tensor [B, R, V] or [N, V], got %s" %
                         (name, _said(t)))
    stride, index = t.stride(), t.get_device()
    if stride[-1] != 1 and shape[-1] != 1:
        raise ValueError("%s: expected a contiguous last dimension, got strides %s" % (name, stride))
    if index != torch.cuda.current_device():
        raise ValueError("%s is on cuda:%d, the current device is cuda:%d" % (name, index, torch.cuda.current_device()))
    if n == 3:
        B, R, V = shape
        return _LOGITS(t.data_ptr(), stride[0], stride[1], B, R, V, dtype), B, R, V, index
    B, V = shape
    return _LOGITS(t.data_ptr(), stride[0], V, B, 1, V, dtype), B, 1, V, index


def _need(name: str, t, shape, dtype, index: int) -> int:
    """The tensor's address, if it is a contiguous one of this shape and type on this GPU."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.shape != shape or t.get_device() != index or \
            not t.is_contiguous():
        raise ValueError("%s: expected a contiguous %s tensor on cuda:%d of shape %s, got %s" %
                         (name, dtype, index, tuple(shape), _said(t)))
    return t.data_ptr()


def _output(out: dict, name: str, shape, dtype, index: int) -> int:
    """The address of output `name`: the caller's tensor, checked, or a new one."""
    t = out.get(name)
    if t is None:
        t = out[name] = torch.empty(shape, dtype=dtype, device="cuda")
        return t.data_ptr()
    return _need(name, t, shape, dtype, index)


def _known(out: Optional[dict], names: set) -> dict:
    if out is None:
        return {}
    if not names.issuperset(out):
        raise ValueError("out: unknown entries among %s (expected %s)" % (sorted(out), sorted(names)))
    return dict(out)


def _scratch(given: Optional[torch.Tensor], need: int, index: int):
    """(a tensor that holds the scratch while the call is made, its address, its bytes)."""
    if given is None:
        if not need:
            return None, None, 0
        given = torch.empty(need, dtype=torch.uint8, device="cuda")
        return given, given.data_ptr(), need
    if not isinstance(given, torch.Tensor) or given.dtype is not torch.uint8 or given.get_device() != index or \
            not given.is_contiguous():
        raise ValueError("workspace: expected a contiguous uint8 tensor on cuda:%d, got %s" % (index, _said(given)))
    return given, given.data_ptr(), given.numel()


# The current stream's handle of a GPU: by the name that torch's own generated code takes it by where there is one
# (torch.cuda.current_stream() builds a Stream object around it each time).
_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda gpu: torch.cuda.current_stream(gpu).cuda_stream)


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
    lib = _declared or _lib()
    lg, B, R, V, gpu = _logits("logits", logits)
    need = top_logits_workspace_size(B, R, V, k, logits.dtype)
    lead = logits.shape[:-1]
    out = _known(out, _TOP_OUT)
    ids = _output(out, "ids", lead + (k,), torch.int32, gpu)
    values = _output(out, "values", lead + (k,), torch.float32, gpu)
    lse = _output(out, "lse", lead, torch.float32, gpu)
    rows = None if n_rows is None else _need("n_rows", n_rows, (B,), torch.int32, gpu)
    _ws, ws, ws_bytes = _scratch(workspace, need, gpu)
    _check(lib.domino_top_logits(lg, k, temperature, rows, ws, ws_bytes, ids, values, lse, _stream(gpu)))
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
    lib = _declared or _lib()
    lg, B, W, V, gpu = _logits("logits", logits)
    if logits.dim() != 3:
        raise ValueError("logits must be [B, W, V]")
    M = W if n_out is None else n_out
    need = beam_step_workspace_size(B, W, V, M, logits.dtype)
    out = _known(out, _BEAM_OUT)
    one = (B, M)
    i_scores = _need("scores", scores, (B, W), torch.float32, gpu)
    o_scores = _output(out, "scores", one, torch.float32, gpu)
    o_parent = _output(out, "parent", one, torch.int32, gpu)
    o_token = _output(out, "token", one, torch.int32, gpu)
    i_finished = i_state = i_history = o_finished = o_state = o_history = state_bytes = T = 0
    if finished is not None:
        i_finished = _need("finished", finished, (B, W), torch.bool, gpu)
    if eos >= 0:
        o_finished = _output(out, "finished", one, torch.bool, gpu)
    if state is not None:
        if not isinstance(state, torch.Tensor) or state.dim() < 2:
            raise ValueError("state must be [B, W, ...]")
        rest = state.shape[2:]
        i_state = _need("state", state, (B, W) + rest, state.dtype, gpu)
        o_state = _output(out, "state", one + rest, state.dtype, gpu)
        state_bytes = rest.numel() * state.element_size()
    if history is not None:
        if not isinstance(history, torch.Tensor) or history.dim() != 3:
            raise ValueError("history must be [B, W, T]")
        T = history.shape[2]
        i_history = _need("history", history, (B, W, T), torch.int32, gpu)
        o_history = _output(out, "history", (B, M, T), torch.int32, gpu)
    if len(out) != 3 + (eos >= 0) + (state is not None) + (history is not None):
        raise ValueError("out: finished needs eos, state and history need their inputs (got %s)" % sorted(out))
    if B and (o_scores == i_scores or (o_state and o_state == i_state) or (o_history and o_history == i_history) or
              (o_finished and o_finished == i_finished)):
        raise ValueError("out: an output tensor is the input it is made from")
    bm = _BEAM(M, eos, T, step, state_bytes, i_scores, i_finished, i_state, i_history, o_scores, o_parent, o_token,
               o_finished, o_state, o_history)
    _ws, ws, ws_bytes = _scratch(workspace, need, gpu)
    _check(lib.domino_beam_step(lg, bm, ws, ws_bytes, _stream(gpu)))
    return out


def distill(logits: torch.Tensor, ids: torch.Tensor, values: torch.Tensor, teacher_lse: Optional[torch.Tensor] = None,
            temperature: float = 1.0, n_rows: Optional[torch.Tensor] = None, grad_loss: Optional[torch.Tensor] = None,
            workspace: Optional[torch.Tensor] = None, out: Optional[dict] = None, want_stats: bool = True) -> dict:
    """Loss of the student's rows against a teacher's top logits, and with `grad_loss` its gradient.

    logits [B, R, V] (or [N, V]) of the student; ids int32 and values float32 [B, R, k] of the teacher
    (`top_logits`); teacher_lse [B, R] float32 at the same temperature: the mass of all other ids is then one
    more event, without it the teacher is its entries alone.  n_rows [B] int32: rows r >= n_rows[b] are left
    out (loss and gradient 0).

    Returns loss [B, R] float32 (temperature^2 times the divergence).  Without grad_loss also stats
    [B, R, 4 + k] float32 for `distill_backward` (want_stats=False, where no gradient follows: the loss alone,
    read past the caches); with grad_loss [B, R] float32 instead grad = grad_loss * dloss/dlogits, of the
    logits' shape and type.  ``out`` may supply these tensors (grad may be the logits
    themselves, or any tensor of their shape and type with a contiguous last dimension), ``workspace`` (uint8)
    the scratch.

    No graph is recorded: the gradient is the one this call or `distill_backward` returns, so without grad_loss
    logits that require one are refused (under no_grad they are taken).  The teacher's entries are constants.
    teacher_lse is a float32: include/domino_head.h says what that leaves open at low temperatures.
    """
    lib = _declared or _lib()
    lg, B, R, V, gpu = _logits("logits", logits)
    lead = logits.shape[:-1]
    k, i_ids = _teacher_ids(ids, lead, gpu)
    need = distill_workspace_size(B, R, V, k, logits.dtype)
    i_values = _need("values", values, lead + (k,), torch.float32, gpu)
    i_lse = None if teacher_lse is None else _need("teacher_lse", teacher_lse, lead, torch.float32, gpu)
    rows = None if n_rows is None else _need("n_rows", n_rows, (B,), torch.int32, gpu)
    i_grad = stats = gd = None
    if grad_loss is None:
        if logits.requires_grad and torch.is_grad_enabled():
            raise ValueError("logits require a gradient, of which the loss records nothing: give grad_loss, or "
                             "logits.detach() and call distill_backward")
        out = _known(out, _LOSS_OUT if want_stats else _LOSS_ONLY)
        if want_stats:
            stats = _output(out, "stats", lead + (STAT_HEAD + k,), torch.float32, gpu)
    else:
        i_grad = _need("grad_loss", grad_loss, lead, torch.float32, gpu)
        out = _known(out, _GRAD_OUT)
        if out.get("grad") is None:
            out["grad"] = torch.empty(logits.shape, dtype=logits.dtype, device="cuda")
        gd = _grad("out['grad']", out["grad"], logits)
    loss = _output(out, "loss", lead, torch.float32, gpu)
    _ws, ws, ws_bytes = _scratch(workspace, need, gpu)
    _check(lib.domino_distill(lg, k, i_ids, i_values, i_lse, temperature, rows, ws, ws_bytes, loss, stats,
                              i_grad, gd, _stream(gpu)))
    return out


def distill_backward(logits: torch.Tensor, ids: torch.Tensor, stats: torch.Tensor, grad_loss: torch.Tensor,
                     temperature: float = 1.0, n_rows: Optional[torch.Tensor] = None,
                     out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """grad_loss * dloss/dlogits of an earlier `distill` call, from its logits, ids and stats.

    grad_loss [B, R] float32; temperature and n_rows as in that call.  ``out`` may be the logits themselves, or
    any tensor of their shape and type with a contiguous last dimension.
    """
    lib = _declared or _lib()
    lg, B, _, _, gpu = _logits("logits", logits)
    lead = logits.shape[:-1]
    k, i_ids = _teacher_ids(ids, lead, gpu)
    i_stats = _need("stats", stats, lead + (STAT_HEAD + k,), torch.float32, gpu)
    i_grad = _need("grad_loss", grad_loss, lead, torch.float32, gpu)
    rows = None if n_rows is None else _need("n_rows", n_rows, (B,), torch.int32, gpu)
    if out is None:
        out = torch.empty(logits.shape, dtype=logits.dtype, device="cuda")
    _check(lib.domino_distill_backward(lg, k, i_ids, i_stats, i_grad, temperature, rows, _grad("out", out, logits),
                                       _stream(gpu)))
    return out


def _teacher_ids(ids, lead, gpu: int):
    if not isinstance(ids, torch.Tensor) or ids.dim() != len(lead) + 1:
        raise ValueError("ids: expected a tensor of shape %s, got %s" % (tuple(lead) + ("k",), _said(ids)))
    k = ids.shape[-1]
    return k, _need("ids", ids, lead + (k,), torch.int32, gpu)


def _grad(name: str, grad, logits: torch.Tensor) -> bytes:
    gd = _logits(name, grad)[0]
    if grad.shape != logits.shape or grad.dtype is not logits.dtype:
        raise ValueError("%s: expected a %s tensor on %s of shape %s, got %s" %
                         (name, logits.dtype, logits.device, tuple(logits.shape), _said(grad)))
    return gd
