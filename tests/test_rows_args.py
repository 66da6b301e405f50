"""Refusals of the operators over vocabulary rows: every host-side check answers before any device work (the
pointers here are never followed), and the Python functions refuse what is not on a GPU."""
import ctypes

import pytest
import torch

import causal_draft_correction_amd as dca
from causal_draft_correction_amd.rows import Beam, Logits, _lib

EINVAL, EUNSUPPORTED, EWORKSPACE = -1, -2, -3
BIG = 1 << 40


def lg(data=16, B=2, R=3, V=100, bs=300, rs=100, dtype=dca.DOMINO_F32):
    return Logits(data, bs, rs, B, R, V, dtype)


def top(x, k=5, tau=1.0, n_rows=None, ws=256, nbytes=BIG, ids=16, values=32, lse=48):
    return _lib().domino_top_logits(ctypes.byref(x), k, tau, n_rows, ws, nbytes, ids, values, lse, None)


def beam(x, ws=256, nbytes=BIG, **kw):
    base = dict(n_out=4, eos=-1, T=0, step=0, state_bytes=0, scores=16, out_scores=32, out_parent=48, out_token=64)
    base.update(kw)
    return _lib().domino_beam_step(ctypes.byref(x), ctypes.byref(Beam(**base)), ws, nbytes, None)


def distill(x, k=5, ids=16, values=32, lse=None, tau=1.0, n_rows=None, ws=256, nbytes=BIG, loss=48, stats=None,
            grad_loss=None, grad=None):
    return _lib().domino_distill(ctypes.byref(x), k, ids, values, lse, tau, n_rows, ws, nbytes, loss, stats, grad_loss,
                                 None if grad is None else ctypes.byref(grad), None)


def backward(x, k=5, ids=16, stats=32, grad_loss=48, tau=1.0, n_rows=None, grad=None):
    return _lib().domino_distill_backward(ctypes.byref(x), k, ids, stats, grad_loss, tau, n_rows,
                                          ctypes.byref(lg(data=4096) if grad is None else grad), None)


SHAPES = [(dict(B=-1), EINVAL), (dict(R=0), EINVAL), (dict(V=0), EINVAL), (dict(dtype=7), EUNSUPPORTED),
          (dict(bs=-1), EINVAL), (dict(rs=-1), EINVAL), (dict(bs=2 ** 62), EINVAL),
          (dict(rs=2 ** 62), EINVAL), (dict(B=2 ** 20, R=2 ** 20), EUNSUPPORTED),
          (dict(B=2 ** 12, R=2 ** 11, V=500000), EUNSUPPORTED),
          (dict(B=2 ** 22, R=4), EUNSUPPORTED), (dict(data=None), EINVAL), (dict(data=18), EINVAL)]


@pytest.mark.parametrize("kw,code", SHAPES)
def test_shapes_types_and_addresses(kw, code):
    for call in (top, beam, distill, backward):
        assert call(lg(**kw)) == code, (call.__name__, kw)
        assert _lib().domino_last_error() != b""


@pytest.mark.parametrize("kw,code", [
    (dict(k=0), EINVAL), (dict(k=129), EINVAL), (dict(tau=0.0), EINVAL), (dict(tau=-1.0), EINVAL),
    (dict(tau=float("nan")), EINVAL), (dict(tau=float("inf")), EINVAL), (dict(tau=1e-5), EINVAL),
    (dict(ids=None), EINVAL), (dict(ids=20), EINVAL), (dict(n_rows=20), EINVAL)])
def test_arguments_of_top_logits_and_distill(kw, code):
    wide = lg(V=1000, rs=1000, bs=3000)
    assert top(wide, **kw) == code
    assert distill(wide, **kw) == code
    assert backward(wide, grad=lg(data=4096, V=1000, rs=1000, bs=3000), **kw) == code


def test_arguments_of_top_logits():
    assert top(lg(V=4, rs=4, bs=12), k=5) == EINVAL
    assert top(lg(V=2 ** 19 + 1)) == EUNSUPPORTED
    for name in ("values", "lse"):
        assert top(lg(), **{name: None}) == EINVAL and top(lg(), **{name: 8}) == EINVAL
    wide = lg(V=40000, rs=40000, bs=120000)
    assert top(wide, ws=None) == EINVAL and top(wide, ws=8) == EINVAL
    need = dca.top_logits_workspace_size(2, 3, 40000, 5)
    assert need > 0 and top(wide, nbytes=need - 1) == EWORKSPACE
    assert b"workspace" in _lib().domino_last_error()
    assert top(lg(B=0, data=None), ws=None, ids=None) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(n_out=0), EINVAL), (dict(n_out=129), EINVAL), (dict(eos=-2), EINVAL), (dict(eos=100), EINVAL),
    (dict(finished=80), EINVAL), (dict(history=80, T=4, step=4, out_history=96), EINVAL),
    (dict(history=80, T=4, step=-1, out_history=96), EINVAL), (dict(history=80, T=0, step=0, out_history=96), EINVAL),
    (dict(history=80, T=4, step=0), EINVAL), (dict(state=80, state_bytes=6, out_state=96), EINVAL),
    (dict(state=80, state_bytes=0, out_state=96), EINVAL), (dict(state=80, state_bytes=8), EINVAL),
    (dict(scores=None), EINVAL), (dict(out_scores=None), EINVAL), (dict(out_parent=None), EINVAL),
    (dict(out_token=None), EINVAL), (dict(scores=24), EINVAL), (dict(out_token=24), EINVAL),
    (dict(eos=1, out_finished=24), EINVAL), (dict(state=88, state_bytes=8, out_state=96), EINVAL)])
def test_arguments_of_beam_step(kw, code):
    assert beam(lg(), **kw) == code


def test_limits_of_beam_step():
    assert beam(lg(B=2 ** 22, R=1, bs=100)) == EUNSUPPORTED
    assert beam(lg(R=33)) == EUNSUPPORTED and beam(lg(V=2 ** 19 + 1)) == EUNSUPPORTED
    assert beam(lg(R=1, V=3), n_out=4) == EINVAL
    need = dca.beam_step_workspace_size(2, 3, 100, 4)
    assert beam(lg(), nbytes=need - 1) == EWORKSPACE and beam(lg(), ws=None) == EINVAL
    assert beam(lg(B=0, data=None), ws=None, scores=None) == 0
    assert _lib().domino_beam_step(ctypes.byref(lg()), None, 256, BIG, None) == EINVAL
    for fn in (top, beam, distill, backward):
        assert fn(lg(B=0)) == 0 or fn is backward  # (backward's gradient has another B)


@pytest.mark.parametrize("kw", [
    dict(grad_loss=80), dict(grad=lg(data=4096)), dict(grad_loss=80, grad=lg(data=4096), stats=64),
    dict(grad_loss=80, grad=lg(data=4096, V=99)), dict(grad_loss=80, grad=lg(data=4096, B=1)),
    dict(grad_loss=80, grad=lg(data=4096, R=2)), dict(grad_loss=80, grad=lg(data=4096, dtype=dca.DOMINO_BF16)),
    dict(grad_loss=80, grad=lg(data=None)), dict(grad_loss=80, grad=lg(data=4098)),
    dict(grad_loss=80, grad=lg(data=4096, rs=99)), dict(grad_loss=80, grad=lg(data=4096, bs=299)),
    dict(grad_loss=80, grad=lg(data=4096, bs=0)), dict(grad_loss=80, grad=lg(data=4096, rs=0)),
    dict(grad_loss=80, grad=lg(data=16, rs=200, bs=600)), dict(grad_loss=72, grad=lg(data=4096)),
    dict(values=None), dict(loss=None), dict(values=24), dict(loss=24), dict(lse=24), dict(stats=24)])
def test_arguments_of_distill(kw):
    assert distill(lg(), **kw) == EINVAL


def test_workspace_of_distill_and_arguments_of_backward():
    wide = lg(V=40000, rs=40000, bs=120000)
    need = dca.distill_workspace_size(2, 3, 40000, 5)
    assert need > 0 and distill(wide, nbytes=need - 1) == EWORKSPACE
    assert distill(wide, ws=None) == EINVAL and distill(wide, ws=24) == EINVAL
    # rows that one block takes whole need none
    assert dca.distill_workspace_size(2, 3, 100, 5) == dca.top_logits_workspace_size(2, 3, 100, 5) == 0
    for kw in (dict(stats=None), dict(grad_loss=None), dict(stats=24), dict(grad_loss=24),
               dict(grad=lg(data=4096, V=99)), dict(grad=lg(data=16, rs=200, bs=600))):
        assert backward(lg(), **kw) == EINVAL
    assert backward(lg(B=0, data=None), grad=lg(B=0, data=None)) == 0


def test_workspace_sizes():
    n = ctypes.c_size_t()
    for fn, args in ((_lib().domino_top_logits_workspace_size, (5,)), (_lib().domino_beam_step_workspace_size, (4,)),
                     (_lib().domino_distill_workspace_size, (5,))):
        assert fn(ctypes.byref(lg()), *args, None) == EINVAL
        assert fn(None, *args, ctypes.byref(n)) == EINVAL
        assert fn(ctypes.byref(lg(B=0)), *args, ctypes.byref(n)) == 0 and n.value == 0
    # the candidates of every chunk fit the list that joins them, at every length and k
    for V in (1, 100, 1024, 5003, 151936, 2 ** 19):
        for k in (1, 5, 127, 128):
            if k <= V:
                for dt in (torch.float32, torch.bfloat16):
                    assert dca.top_logits_workspace_size(1, 1, V, k, dt) <= (4096 + 128) * 8 + 4096 * 8 + 48
    with pytest.raises(dca.DominoError):
        dca.top_logits_workspace_size(1, 1, 2 ** 19 + 1, 1)
    with pytest.raises(ValueError):
        dca.top_logits_workspace_size(1, 1, 100, 1, torch.float16)


def test_python_functions_refuse_host_tensors():
    z = torch.zeros((1, 2, 10))
    ids, values, one = torch.zeros((1, 2, 3), dtype=torch.int32), torch.zeros((1, 2, 3)), torch.zeros((1, 2))
    for call in (lambda: dca.top_logits(z, 3), lambda: dca.beam_step(z, one), lambda: dca.distill(z, ids, values),
                 lambda: dca.distill_backward(z, ids, torch.zeros((1, 2, 7)), one), lambda: dca.top_logits(None, 3)):
        with pytest.raises(ValueError, match="logits"):
            call()
