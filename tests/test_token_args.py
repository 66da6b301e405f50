"""Refusals of the token log-probabilities: every host-side check answers before any device work (the pointers here are
never followed)."""
import ctypes

import pytest
import torch

import causal_draft_correction_amd as dca
from causal_draft_correction_amd.rows import Logits, _lib
from test_rows_args import SHAPES, lg

EINVAL, EUNSUPPORTED, EWORKSPACE, EHIP = -1, -2, -3, -4
BIG = 1 << 40
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="would launch on these pointers if it were not refused")


def at(n):
    """Pointers 64 KiB apart, away from the logits."""
    return (2 << 20) + (n << 16)


def ref(x):
    return None if x is None else ctypes.byref(x)


def score(x, k=0, tokens=at(0), tau=1.0, n_rows=None, ws=at(9), nbytes=BIG, logprob=at(1), entropy=at(2), ids=None,
          logprobs=None, stats=None, g1=None, g2=None, grad=None):
    if k and ids is None:
        ids, logprobs = at(3), at(4)
    return _lib().domino_token_logprobs(ref(x), tokens, k, tau, n_rows, ws, nbytes, logprob, entropy, ids or None,
                                        logprobs, stats, g1, g2, ref(grad), None)


def back(x, grad, tokens=at(0), stats=at(5), g1=at(6), g2=None, tau=1.0, n_rows=None):
    return _lib().domino_token_logprobs_backward(ref(x), tokens, stats, g1, g2, tau, n_rows, ref(grad), None)


DATA = 1 << 20
GRAD = DATA + 4096


@pytest.mark.parametrize("kw,code", SHAPES)
def test_shapes_types_and_addresses(kw, code):
    assert score(lg(**kw)) == score(lg(**kw), k=3) == back(lg(**kw), lg(data=GRAD)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(k=-1), EINVAL), (dict(k=129), EINVAL), (dict(k=101), EINVAL), (dict(tau=0.0), EINVAL), (dict(tau=1e5), EINVAL),
    (dict(tau=float("nan")), EINVAL), (dict(tokens=None), EINVAL), (dict(tokens=at(0) + 4), EINVAL),
    (dict(n_rows=24), EINVAL), (dict(logprob=None), EINVAL), (dict(entropy=None), EINVAL), (dict(logprob=24), EINVAL),
    (dict(entropy=24), EINVAL), (dict(k=3, ids=20), EINVAL), (dict(k=3, ids=at(3), logprobs=None), EINVAL),
    (dict(k=0, ids=at(3), logprobs=at(4)), EINVAL), (dict(stats=24), EINVAL), (dict(g1=at(6)), EINVAL),
    (dict(grad=lg(data=GRAD)), EINVAL), (dict(g1=at(6), grad=lg(data=GRAD), stats=at(5)), EINVAL),
    (dict(g1=at(6), grad=lg(data=GRAD), k=2), EINVAL), (dict(g1=24, grad=lg(data=GRAD)), EINVAL),
    (dict(g2=24, grad=lg(data=GRAD)), EINVAL), (dict(g2=at(6), grad=lg(data=GRAD, V=99)), EINVAL),
    (dict(g2=at(6), grad=lg(data=GRAD, rs=99)), EINVAL), (dict(g2=at(6), grad=lg(data=None)), EINVAL)])
def test_arguments(kw, code):
    assert score(lg(data=DATA), **kw) == code


def test_backward_workspaces_and_limits():
    for kw in (dict(tokens=None), dict(stats=None), dict(g1=None), dict(g1=24), dict(stats=24), dict(tau=0.0)):
        assert back(lg(data=DATA), lg(data=GRAD), **kw) == EINVAL
    wide = lg(V=40000, rs=40000, bs=120000)
    for k in (0, 5):
        need = dca.token_logprobs_workspace_size(2, 3, 40000, k)
        assert need > 0 and need % 16 == 0 and score(wide, k=k, nbytes=need - 1) == EWORKSPACE
        assert score(wide, k=k, ws=None) == score(wide, k=k, ws=24) == EINVAL
    assert dca.token_logprobs_workspace_size(2, 3, 100) == dca.token_logprobs_workspace_size(2, 3, 100, 100) == 0
    long = lg(V=2 ** 19 + 1, rs=2 ** 20, bs=2 ** 22)
    assert score(long, k=3) == EUNSUPPORTED
    assert score(lg(B=0, data=None), tokens=None, logprob=None, ws=None) == 0
    assert _lib().domino_token_logprobs_workspace_size(ref(lg()), 0, None) == EINVAL
    assert score(None) == back(None, lg()) == back(lg(data=DATA), None) == EINVAL


@no_gpu
def test_memory_shared_by_the_arguments():
    def refused(code):
        return code == EINVAL and b"overlaps" in _lib().domino_last_error()

    x = lg(data=DATA)
    for kw in (dict(logprob=at(0)), dict(entropy=at(1)), dict(logprob=DATA + 16), dict(stats=at(0)), dict(stats=at(2)),
               dict(k=5, ids=at(4), logprobs=at(4)), dict(k=5, ids=DATA, logprobs=at(4)),
               dict(k=5, ids=at(3), logprobs=at(0) - 112), dict(g1=at(1), grad=lg(data=GRAD)),
               dict(g1=GRAD, grad=lg(data=GRAD)), dict(g2=at(6), logprob=GRAD + 16, grad=lg(data=GRAD)),
               dict(g2=at(6), grad=lg(data=DATA + 400))):
        assert refused(score(x, **kw)), kw
    wide = lg(data=DATA, V=40000, rs=40000, bs=120000)
    far = 1 << 30
    for kw in (dict(ws=DATA), dict(ws=far, logprob=far)):
        assert refused(score(wide, tokens=far + (1 << 20), **{**dict(logprob=far + (2 << 20), entropy=far + (3 << 20)), **kw}))
    for kw in (dict(tokens=GRAD), dict(stats=GRAD + 16), dict(g1=GRAD)):
        assert refused(back(x, lg(data=GRAD), **kw)), kw
    assert score(x) == score(x, k=5) == score(x, g1=at(6), grad=lg(data=GRAD)) == EHIP
    assert score(x, g1=at(6), grad=x) == back(x, x) == back(x, lg(data=DATA + 2400)) == EHIP  # in place, and beside it
