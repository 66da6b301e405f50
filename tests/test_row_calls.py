"""Calls of the operators over vocabulary rows as the host sees them: what the package needs of torch when it is
imported, workspaces, and refusals (the pointers here are never followed)."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

import causal_draft_correction_amd as dca
from causal_draft_correction_amd.rows import Beam, Logits, _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
EINVAL, EUNSUPPORTED, EWORKSPACE = -1, -2, -3


def test_the_package_imports_without_the_private_stream_name():
    code = ("import torch\n"
            "if hasattr(torch._C, '_cuda_getCurrentRawStream'):\n"
            "    del torch._C._cuda_getCurrentRawStream\n"
            "import causal_draft_correction_amd as dca\n"
            "from causal_draft_correction_amd import rows\n"
            "class One:\n"
            "    cuda_stream = 7\n"
            "torch.cuda.current_stream = lambda gpu: One\n"
            "assert rows._stream(0) == 7 and dca.top_logits is rows.top_logits\n")
    got = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert got.returncode == 0, got.stderr


# ---- memory that outputs share with what a call reads or writes besides ----

def lg(data=1 << 20, B=2, R=3, V=100, bs=300, rs=100, dtype=dca.DOMINO_F32):
    return Logits(data, bs, rs, B, R, V, dtype)


def at(n, off=0):
    """The n-th of pointers 64 KiB apart, away from the logits."""
    return (2 << 20) + (n << 16) + off


def top(x, ids=at(0), values=at(1), lse=at(2), n_rows=None, ws=at(3), k=5):
    return _lib().domino_top_logits(ctypes.byref(x), k, 1.0, n_rows, ws, 1 << 30, ids, values, lse, None)


def beam(x, ws=at(15), **kw):
    base = dict(n_out=4, eos=1, T=8, step=0, state_bytes=64, scores=at(0), finished=at(1), state=at(2), history=at(3),
                out_scores=at(4), out_parent=at(5), out_token=at(6), out_finished=at(7), out_state=at(8),
                out_history=at(9))
    base.update(kw)
    return _lib().domino_beam_step(ctypes.byref(x), ctypes.byref(Beam(**base)), ws, 1 << 30, None)


def distill(x, grad=None, ids=at(0), values=at(1), lse=at(2), n_rows=at(3), loss=at(4), stats=None, grad_loss=at(6),
            ws=at(7)):
    return _lib().domino_distill(ctypes.byref(x), 5, ids, values, lse, 1.0, n_rows, ws, 1 << 30, loss, stats,
                                 grad_loss if grad else None, ctypes.byref(grad) if grad else None, None)


def backward(x, grad, ids=at(0), stats=at(5), grad_loss=at(6)):
    return _lib().domino_distill_backward(ctypes.byref(x), 5, ids, stats, grad_loss, 1.0, None, ctypes.byref(grad),
                                          None)


no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="would launch on these pointers if it were not refused")
DATA = 1 << 20  # the logits' 2400 bytes: rows of 400
WIDE = dict(V=40000, bs=120000, rs=40000)  # split rows, which use the workspace


def refused(code):
    return code == EINVAL and b"overlaps" in _lib().domino_last_error()


@no_gpu
def test_outputs_on_inputs_or_each_other_are_refused():
    for kw in (dict(ids=DATA), dict(ids=DATA + 2384), dict(ids=DATA - 112), dict(values=at(0)), dict(values=at(0, 112)),
               dict(lse=at(1, 112)), dict(n_rows=at(2, 16)), dict(n_rows=at(0))):
        assert refused(top(lg(), **kw)), kw
    for kw in (dict(ws=at(0)), dict(ws=DATA), dict(ws=at(1, 112)), dict(n_rows=at(3, 16))):
        assert refused(top(lg(**WIDE), **kw)), kw
        assert refused(distill(lg(**WIDE), ws=at(4), **{n: v for n, v in kw.items() if n != "ws"}))
    for kw in (dict(out_scores=at(0)), dict(out_scores=at(0, 16)), dict(out_state=at(2, 320)), dict(out_state=at(3)),
               dict(out_history=at(3, 176)), dict(out_parent=at(4, 16)), dict(out_token=at(5)), dict(out_finished=at(1)),
               dict(out_state=at(4)), dict(out_history=at(8, 496)), dict(out_token=DATA + 16), dict(ws=at(0)),
               dict(ws=at(2)), dict(ws=DATA), dict(out_finished=at(8, 496))):
        assert refused(beam(lg(), **kw)), kw
    for kw in (dict(loss=at(0)), dict(loss=at(1, 112)), dict(loss=DATA), dict(stats=at(0)), dict(stats=at(4, 16)),
               dict(stats=DATA + 2384), dict(n_rows=at(4))):
        assert refused(distill(lg(), **kw)), kw


@no_gpu
@pytest.mark.parametrize("data,bs,rs", [
    (DATA + 4, 300, 100), (DATA - 4, 300, 100), (DATA + 400, 300, 100), (DATA + 1200, 300, 100), (DATA + 2396, 300, 100),
    (DATA - 2396, 300, 100), (DATA, 600, 200), (DATA, 100, 200), (DATA + 396, 600, 200), (DATA - 1600, 10 ** 6, 201),
    (DATA + 1, 300, 100)])
def test_gradients_that_overlap_the_logits_are_refused(data, bs, rs):
    grad = lg(data=data, bs=bs, rs=rs)
    for code in (distill(lg(), grad), backward(lg(), grad)):
        assert refused(code) or (data % 4 and code == EINVAL)


@no_gpu
def test_gradients_over_other_arguments_are_refused():
    for kw in (dict(ids=DATA + 8000), dict(values=DATA + 8016), dict(loss=DATA + 10384), dict(grad_loss=DATA + 8000),
               dict(lse=DATA + 8000), dict(n_rows=DATA + 8000)):
        assert refused(distill(lg(), lg(data=DATA + 8000), **kw)), kw
    for kw in (dict(ids=DATA + 8000), dict(stats=DATA + 8016), dict(grad_loss=DATA + 10384)):
        assert refused(backward(lg(), lg(data=DATA + 8000), **kw)), kw


@no_gpu
def test_rows_side_by_side_are_not_refused():
    """What passes every check ends at the launch, which fails without a GPU."""
    EHIP = -4
    assert top(lg()) == beam(lg()) == distill(lg()) == distill(lg(), lg(data=DATA + 2400)) == EHIP
    assert distill(lg(), lg(data=DATA - 2400)) == EHIP
    wide = lg(bs=600, rs=200)  # the gradient in the other half of every row; of every batch entry; rows exchanged
    assert distill(wide, lg(data=DATA + 400, bs=600, rs=200)) == EHIP
    assert backward(wide, lg(data=DATA - 400, bs=600, rs=200)) == EHIP
    assert backward(lg(bs=600), lg(data=DATA + 1200, bs=600)) == EHIP
    assert backward(lg(bs=100, rs=400), lg(data=DATA + 800, bs=100, rs=400)) == EHIP
    assert backward(wide, lg(data=DATA + 400, bs=200, rs=400)) == EHIP
    assert backward(wide, lg(data=DATA + 400, bs=300, rs=600)) == EINVAL  # (its fourth row is the logits' third)
    # outputs between the rows
    assert top(lg(bs=900, rs=300), ids=DATA + 400, values=DATA + 1600, lse=DATA + 2800) == EHIP
    # the logits' own rows: the stride of a dimension of length 1 says nothing
    assert distill(lg(), lg()) == backward(lg(), lg()) == EHIP
    assert distill(lg(B=1), lg(B=1, bs=7)) == EHIP and backward(lg(R=1), lg(R=1, rs=12345)) == EHIP
    assert distill(lg(R=1, bs=0, B=1), lg(R=1, B=1)) == EHIP


@no_gpu
def test_overlaps_of_rows_against_every_byte():
    """All placements of small strided rows, gradient against logits, by the sets of their elements."""
    import itertools
    import random

    rng = random.Random(5)
    for _ in range(4000):
        B, R, V = rng.randint(1, 3), rng.randint(1, 3), rng.randint(1, 4)

        def place():
            while True:
                rs, bs = rng.randint(0, 14), rng.randint(0, 40)
                if rng.random() < 0.3:
                    rs, bs = bs, rs
                return rs, bs

        rs, bs = place()
        grs, gbs = place()
        cells = lambda base, b_s, r_s: [base + b * b_s + r * r_s + v for b, r, v in  # noqa: E731
                                        itertools.product(range(B), range(R), range(V))]
        off = rng.randint(-60, 60)
        x, g = cells(0, bs, rs), cells(off, gbs, grs)
        if len(set(g)) < len(g):
            continue  # (the gradient's own rows)
        got = backward(lg(B=B, R=R, V=V, bs=bs, rs=rs), lg(data=DATA + 4 * off, B=B, R=R, V=V, bs=gbs, rs=grs))
        own = off == 0 and (B == 1 or bs == gbs) and (R == 1 or rs == grs)
        nested = (R == 1 or grs >= V) and (B == 1 or gbs >= V) and \
            (R == 1 or B == 1 or gbs >= (R - 1) * grs + V or grs >= (B - 1) * gbs + V)
        if not nested:
            assert got == EINVAL
        else:
            assert (got == EINVAL) == (bool(set(x) & set(g)) and not own), (B, R, V, bs, rs, off, gbs, grs)


# ---- workspaces ----

@pytest.mark.parametrize("dtype,per", [(torch.float32, 4), (torch.bfloat16, 8)])
def test_candidates_of_all_chunks_fit_the_list_that_joins_them(dtype, per):
    """8 bytes a candidate and at most 4096 of a row, 16 bytes for each of at most 64 chunks."""
    edges = [256 * 8 * per * n + d for n in (1, 2, 3, 4, 5, 8, 16, 17, 31, 32, 33) for d in (-1, 0, 1)]
    lengths = sorted({V for V in edges + [1, 100, 5003, 50021, 151936, 2 ** 19 - 1, 2 ** 19] if 1 <= V <= 2 ** 19})
    for V in lengths:
        for k in (1, 5, 31, 32, 33, 63, 64, 65, 127, 128):
            for B, R in ((1, 1), (1, 2), (1, 17), (3, 20), (255, 1), (16, 16), (257, 1), (64, 16)):
                if k <= V:
                    need = dca.top_logits_workspace_size(B, R, V, k, dtype)
                    rows = B * R
                    assert need % 16 == 0 and need <= rows * (4096 * 8 + 64 * 16) + 32, (V, k, rows)
                    if need:  # chunks of k candidates and a part each
                        assert any(need == (rows * n * k * 8 + 15) // 16 * 16 + rows * n * 16
                                   for n in range(1, 65)), (V, k, rows)
