"""Refusals of the layers: every host-side check answers before any device work (the pointers here are never
followed), and the Python functions refuse what is not on a GPU."""
import ctypes

import pytest
import torch

import causal_draft_correction_amd as dca
from causal_draft_correction_amd.layers import _lib
from causal_draft_correction_amd.rows import Logits as Rows

EINVAL, EUNSUPPORTED, EWORKSPACE, EHIP = -1, -2, -3, -4
BIG = 1 << 40
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="would launch on these pointers if it were not refused")


def rows(data=1 << 20, B=2, R=3, V=100, bs=300, rs=100, dtype=dca.DOMINO_F32):
    return Rows(data, bs, rs, B, R, V, dtype)


def table(data=1 << 24, R=50, V=100, rs=100, B=1, dtype=dca.DOMINO_BF16):
    return Rows(data, 0, rs, B, R, V, dtype)


def ref(x):
    return None if x is None else ctypes.byref(x)


def embed(t, out, ids=16, scale=1.0):
    return _lib().domino_embed(ref(t), ids, scale, ref(out), None)


def backward(grad, t, ids=16, scale=1.0, accumulate=0, ws=256, nbytes=BIG):
    return _lib().domino_embed_backward(ref(grad), ids, scale, accumulate, ws, nbytes, ref(t), None)


SHAPES = [(dict(B=-1), EINVAL), (dict(R=0), EINVAL), (dict(V=0), EINVAL), (dict(dtype=7), EUNSUPPORTED),
          (dict(bs=-1), EINVAL), (dict(rs=-1), EINVAL), (dict(bs=2 ** 62), EINVAL), (dict(V=99), EINVAL),
          (dict(B=2 ** 20, R=2 ** 20), EUNSUPPORTED), (dict(data=None), EINVAL), (dict(data=18), EINVAL)]


@pytest.mark.parametrize("kw,code", SHAPES)
def test_rows_of_an_embedding(kw, code):
    assert embed(table(), rows(**kw)) == code
    assert backward(rows(**kw), table()) == code
    assert _lib().domino_last_error() != b""


@pytest.mark.parametrize("kw,code", [
    (dict(B=2), EINVAL), (dict(B=0), EINVAL), (dict(R=0), EINVAL), (dict(V=101), EINVAL), (dict(dtype=3), EUNSUPPORTED),
    (dict(rs=-4), EINVAL), (dict(data=None), EINVAL), (dict(data=17), EINVAL)])
def test_table_of_an_embedding(kw, code):
    assert embed(table(**kw), rows()) == code
    assert backward(rows(), table(**kw)) == code


def test_other_arguments_of_an_embedding():
    assert embed(table(), None) == embed(None, rows()) == backward(None, table()) == backward(rows(), None) == EINVAL
    for scale in (float("nan"), float("inf"), 1e39):
        assert embed(table(), rows(), scale=scale) == backward(rows(), table(), scale=scale) == EINVAL
    for ids in (None, 18):
        assert embed(table(), rows(), ids=ids) == backward(rows(), table(), ids=ids) == EINVAL
    assert embed(table(), rows(rs=99)) == embed(table(), rows(bs=299)) == embed(table(), rows(rs=0)) == EINVAL
    assert backward(rows(), table(rs=99)) == EINVAL
    wide = 2 ** 20 + 1
    assert embed(table(V=wide, rs=wide), rows(V=wide, rs=wide, bs=3 * wide)) == EUNSUPPORTED
    need = dca.embed_backward_workspace_size(2, 3, 100)
    assert need > 0 and need % 16 == 0
    assert backward(rows(), table(), nbytes=need - 1) == EWORKSPACE
    assert backward(rows(), table(), ws=None) == backward(rows(), table(), ws=24) == EINVAL
    assert embed(table(), rows(B=0, data=None), ids=None) == 0
    assert backward(rows(B=0, data=None), table(data=None), ids=None, accumulate=1, ws=None) == 0
    assert _lib().domino_embed_backward_workspace_size(ref(rows()), None) == EINVAL


@no_gpu
def test_memory_shared_by_an_embeddings_arguments():
    def refused(code):
        return code == EINVAL and b"overlaps" in _lib().domino_last_error()

    at = 1 << 20  # the rows' 2400 bytes
    t = 1 << 24  # the table's 10000
    for out in (rows(data=t), rows(data=t - 2396), rows(data=t + 9996)):
        assert refused(embed(table(), out)) and refused(backward(out, table(), ids=64, ws=256))
    assert refused(embed(table(), rows(), ids=at + 2396)) and refused(embed(table(), rows(), ids=at - 20))
    assert refused(backward(rows(), table(), ids=t)) and refused(backward(rows(), table(), ws=t))
    assert refused(backward(rows(), table(), ids=256, ws=256)) and refused(backward(rows(), table(), ws=at + 16))
    # beside each other
    assert embed(table(), rows(), ids=at + 2400) == embed(table(), rows(data=t - 2400)) == EHIP
    assert embed(table(), rows(data=t + 10000)) == EHIP
    # the table's rows of 200 bytes begin every 800: rows at 200, 600, 1000 ... lie between them, at 300, 700, ... do not
    assert embed(table(rs=400), rows(data=t + 200, rs=200, bs=600, V=100, dtype=dca.DOMINO_BF16)) == EHIP
    assert refused(embed(table(rs=400), rows(data=t + 300, rs=200, bs=600, V=100, dtype=dca.DOMINO_BF16)))
    assert embed(table(rs=400), rows(data=t + 200, rs=400, bs=1200, V=100, dtype=dca.DOMINO_BF16)) == EHIP


def test_python_refuses_what_is_not_on_a_gpu():
    ids = torch.zeros(3, dtype=torch.int32)
    for call in (lambda: dca.embed(torch.zeros(5, 4), ids), lambda: dca.embed(None, ids),
                 lambda: dca.embed_backward(torch.zeros(3, 4), ids, 5), lambda: dca.embed(torch.zeros(5, 4, 2), ids)):
        with pytest.raises(ValueError):
            call()
