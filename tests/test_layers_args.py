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
    need, many = dca.embed_backward_workspace_size(200, 3, 100), rows(B=200)
    assert dca.embed_backward_workspace_size(2, 3, 100) == 0 and need > 0 and need % 16 == 0
    assert backward(many, table(), nbytes=need - 1) == EWORKSPACE
    assert backward(many, table(), ws=None) == backward(many, table(), ws=24) == EINVAL
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
    many = dict(B=200)
    assert refused(backward(rows(), table(), ids=t)) and refused(backward(rows(**many), table(), ws=t))
    assert refused(backward(rows(**many), table(), ids=256, ws=256))
    assert refused(backward(rows(**many), table(), ids=1 << 27, ws=at + 16))
    assert backward(rows(**many), table(), ids=1 << 27, ws=1 << 28) == backward(rows(), table(), ws=None) == EHIP
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


# ---- linear layers ----

def w(data=1 << 24, N=50, K=100, rs=100, B=1, dtype=dca.DOMINO_BF16):
    return Rows(data, 0, rs, B, N, K, dtype)


def y(data=1 << 28, B=2, R=3, V=50, bs=150, rs=50, dtype=dca.DOMINO_F32):
    return Rows(data, bs, rs, B, R, V, dtype)


def linear(x, wt, out, bias=None, act=0, residual=None, ws=256, nbytes=BIG, pre=None):
    return _lib().domino_linear(ref(x), ref(wt), ref(bias), act, ref(residual), ws, nbytes, ref(out), ref(pre), None)


def linear_back(g, x, wt, pre=None, act=0, acc=0, ws=256, nbytes=BIG, dx=None, dw=None, db=None):
    return _lib().domino_linear_backward(ref(g), ref(x), ref(wt), ref(pre), act, acc, ws, nbytes, ref(dx), ref(dw),
                                         ref(db), None)


DX, DW, DB = rows(data=1 << 29), w(data=1 << 30, dtype=dca.DOMINO_F32), Rows(1 << 27, 0, 0, 1, 1, 50, dca.DOMINO_F32)


@pytest.mark.parametrize("kw,code", SHAPES)
def test_rows_of_a_linear_layer(kw, code):
    assert linear(rows(**kw), w(), y()) == code
    assert linear_back(y(), rows(**kw), w(), dw=DW) == code
    assert linear_back(y(), rows(), w(), dx=rows(**{"data": 1 << 29, **kw})) == code
    assert _lib().domino_last_error() != b""


@pytest.mark.parametrize("kw,code", [
    (dict(B=2), EINVAL), (dict(B=0), EINVAL), (dict(N=0), EINVAL), (dict(K=101), EINVAL), (dict(dtype=3), EUNSUPPORTED),
    (dict(rs=-4), EINVAL), (dict(data=None), EINVAL), (dict(data=17), EINVAL), (dict(N=51), EINVAL)])
def test_weights_of_a_linear_layer(kw, code):
    assert linear(rows(), w(**kw), y()) == code
    assert linear_back(y(), rows(), w(**kw), dx=DX) == code
    assert linear_back(y(), rows(), w(), dw=w(**{"data": 1 << 30, **kw})) == code


@pytest.mark.parametrize("kw,code", [
    (dict(B=1), EINVAL), (dict(R=2), EINVAL), (dict(V=49), EINVAL), (dict(dtype=9), EUNSUPPORTED), (dict(rs=-1), EINVAL),
    (dict(data=None), EINVAL), (dict(data=6), EINVAL)])
def test_outputs_of_a_linear_layer(kw, code):
    other = {"data": 1 << 26, **kw}
    for call in (lambda: linear(rows(), w(), y(**kw)), lambda: linear(rows(), w(), y(), pre=y(**other)),
                 lambda: linear(rows(), w(), y(), residual=y(**other)), lambda: linear_back(y(**kw), rows(), w(), dx=DX),
                 lambda: linear_back(y(), rows(), w(), pre=y(**other), act=1, dx=DX)):
        assert call() == code


def test_other_arguments_of_a_linear_layer():
    assert linear(rows(), w(), y(rs=49)) == linear(rows(), w(), y(), pre=y(data=1 << 26, bs=149)) == EINVAL
    assert linear(rows(), w(), None) == linear(None, w(), y()) == linear(rows(), None, y()) == EINVAL
    for act in (-1, 4):
        assert linear(rows(), w(), y(), act=act) == linear_back(y(), rows(), w(), act=act, dx=DX) == EINVAL
    assert linear_back(y(), rows(), w()) == EINVAL
    assert linear_back(y(), rows(), w(), act=1, dx=DX) == EINVAL  # (without pre)
    assert linear_back(y(), rows(), w(), pre=y(data=1 << 26), dx=DX) == EINVAL
    for bias in (Rows(64, 0, 0, 1, 1, 49, 0), Rows(64, 0, 0, 1, 2, 50, 0), Rows(None, 0, 0, 1, 1, 50, 0)):
        assert linear(rows(), w(), y(), bias=bias) == linear_back(y(), rows(), w(), db=bias) == EINVAL
    far, many = 1 << 40, 1 << 17  # 2^17 rows of 2^16: too many for gelu alone
    huge = [rows(B=many, R=1, V=8, bs=8, rs=8), Rows(far, 0, 8, 1, 1 << 16, 8, 0), y(data=1 << 41, B=many, R=1, V=1 << 16,
                                                                                   bs=1 << 16)]
    assert linear(*huge, act=2) == EUNSUPPORTED
    long = 1 << 24
    assert linear(rows(V=long, rs=long, bs=3 * long, B=1, R=1), w(K=long, rs=long, N=1), y(B=1, R=1, V=1)) == EUNSUPPORTED
    need = dca.linear_workspace_size(2, 3, 5000, 50)
    wide = rows(V=5000, rs=5000, bs=15000), w(K=5000, rs=5000)
    assert need > 0 and linear(*wide, y(), nbytes=need - 1) == EWORKSPACE
    assert linear(*wide, y(), ws=None) == linear(*wide, y(), ws=24) == EINVAL
    need = dca.linear_backward_workspace_size(2, 3, 100, 50, "silu")
    pre = y(data=1 << 26)
    assert need > 0 and linear_back(y(), rows(), w(), pre=pre, act=1, dx=DX, nbytes=need - 1) == EWORKSPACE
    assert linear(rows(B=0, data=None), w(), y(B=0, data=None), ws=None) == 0
    assert _lib().domino_linear_workspace_size(ref(rows()), ref(w()), 0, None) == EINVAL
    assert _lib().domino_linear_backward_workspace_size(ref(y()), ref(rows()), ref(w()), 0, 1, 1, 1, None) == EINVAL


@no_gpu
def test_memory_shared_by_a_linear_layers_arguments():
    def refused(code):
        return code == EINVAL and b"overlaps" in _lib().domino_last_error()

    x, wt, out = rows(), w(), y()
    bias = Rows(1 << 27, 0, 0, 1, 1, 50, dca.DOMINO_F32)
    residual, pre = y(data=1 << 26), y(data=1 << 25)
    assert linear(x, wt, out, bias=bias, residual=residual, pre=pre, act=1) == EHIP
    for data in (1 << 20, (1 << 20) + 2396, (1 << 24) - 1196, 1 << 27, 1 << 25, (1 << 26) + 600):
        assert refused(linear(x, wt, y(data=data), bias=bias, residual=residual, pre=pre, act=1)), data
    assert refused(linear(x, wt, out, residual=residual, pre=residual))
    assert refused(linear(x, wt, out, pre=out))
    assert linear(x, wt, out, residual=out) == EHIP  # in its place
    assert refused(linear(x, wt, out, residual=y(dtype=dca.DOMINO_BF16))) and refused(linear(x, wt, out, residual=y(rs=51)))
    wide = rows(V=5000, rs=5000, bs=15000), w(K=5000, rs=5000)
    assert refused(linear(*wide, out, ws=1 << 28)) and refused(linear(*wide, out, ws=1 << 24))
    kw = dict(pre=pre, act=1, dx=DX, dw=DW, db=DB)
    assert linear_back(out, x, wt, **kw) == EHIP
    for name, one in (("dx", rows(data=1 << 20)), ("dx", rows(data=(1 << 24) - 2396)), ("dx", rows(data=1 << 30)),
                      ("dw", w(data=(1 << 29) + 16)), ("dw", w(data=1 << 28)), ("db", Rows(1 << 25, 0, 0, 1, 1, 50, 0)),
                      ("db", Rows((1 << 30) + 64, 0, 0, 1, 1, 50, 0)), ("dw", w())):
        assert refused(linear_back(out, x, wt, **{**kw, name: one})), name
    assert refused(linear_back(out, x, wt, ws=1 << 29, **kw)) and refused(linear_back(out, x, wt, ws=1 << 25, **kw))


def test_python_refuses_layers_that_are_not_on_a_gpu():
    x, wt, g = torch.zeros(3, 4), torch.zeros(5, 4), torch.zeros(3, 5)
    for call in (lambda: dca.linear(x, wt), lambda: dca.linear_backward(g, x, wt), lambda: dca.linear(None, wt)):
        with pytest.raises(ValueError):
            call()
