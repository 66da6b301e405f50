"""GPU results of the embedding and its gradient against their plain 64-bit forms (layers_plain.py).

Bounds, in halves of a float32 step (H = 2^-24).  A looked-up element is one product, rounded to float32 (H) and to the
output's type.  A token's gradient adds its n rows in turn (up to 256 tokens), or in tiles of at most 64, the tiles' sums in 16
strands and these in turn: of n float32 additions an addend passes through at most max(256, 64 + n / 256 + 17) (and no
more than n), each of which rounds a value no larger than the sum of magnitudes; the scale and the addition to an earlier gradient round once more
each; then the output's type."""
import numpy as np
import pytest
import torch

import causal_draft_correction_amd as dca
import layers_plain as plain

pytestmark = pytest.mark.gpu

H = 2.0 ** -24
HALF = {torch.float32: H, torch.bfloat16: 2.0 ** -8}
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dca.load_library()


def host(t):
    return t.float().cpu().numpy()


def matrix(rows, cols, dtype, seed, pad=0, shift=0):
    """[rows, cols], a view of a buffer with `pad` columns after each row and `shift` elements before the first."""
    g = torch.Generator().manual_seed(seed)
    flat = torch.randn(shift + rows * (cols + pad), generator=g).to(dtype).cuda()
    return flat[shift:].view(rows, cols + pad)[:, :cols]


def tokens(n, V, kind, seed):
    g = torch.Generator().manual_seed(seed)
    if kind == "one":
        ids = torch.full((n,), V // 2)
    elif kind == "even":
        ids = torch.randint(0, V, (n,), generator=g)
    elif kind == "few":  # runs of any length against the tiles'
        ids = torch.randint(0, 7, (n,), generator=g) * (V - 1) // 6
    elif kind == "outside":
        ids = torch.randint(-V, 2 * V, (n,), generator=g)
    elif kind == "none":
        ids = torch.where(torch.rand(n, generator=g) < 0.5, -1, V)
    else:  # zipf
        ids = torch.exp(torch.rand(n, generator=g) * np.log(V)).long().clamp(1, V) - 1
    return ids.int().cuda()


@pytest.mark.parametrize("ttype,otype", [(F32, F32), (F32, BF16), (BF16, F32), (BF16, BF16)])
@pytest.mark.parametrize("n,V,d,pad,shift,scale", [
    (1, 1, 1, 0, 0, 1.0), (3, 10, 7, 1, 1, 0.3), (17, 100, 64, 0, 0, 2.0), (1000, 333, 1031, 3, 5, -1.7),
    (5, 50, 4096, 0, 3, 64.0), (257, 9, 8, 8, 0, 0.0)])
def test_embed(n, V, d, pad, shift, scale, ttype, otype):
    table, ids = matrix(V, d, ttype, n + d, pad, shift), tokens(n, V, "outside", n)
    out = matrix(n, d, otype, 1, 2 * pad, shift)
    keep = out.storage_offset(), out.stride()
    wide = torch.as_strided(out, (out.untyped_storage().nbytes() // out.element_size(),), (1,), 0)
    before = wide.clone()
    dca.embed(table, ids, scale=scale, out=out)
    assert (out.storage_offset(), out.stride()) == keep
    want = plain.embed(host(table), ids.cpu().numpy(), float(np.float32(scale)))
    bound = np.abs(want) * (H + HALF[otype] * (1 + H)) + 2.0 ** -140
    assert (np.abs(host(out) - want) <= bound).all()
    mask = torch.ones_like(wide, dtype=torch.bool)
    torch.as_strided(mask, out.shape, out.stride(), out.storage_offset()).fill_(False)
    assert torch.equal(wide[mask].view(torch.uint8), before[mask].view(torch.uint8))  # nothing beside the rows
    assert torch.equal(dca.embed(table, ids, scale=scale).float(), dca.embed(table, ids.view(1, -1), scale=scale)[0].float())


def check_backward(grad, ids, V, scale, otype, accumulate=False, pad=0, shift=0, label=""):
    d = grad.shape[-1]
    out = matrix(V, d, otype, 5, pad, shift)
    was = host(out).astype(np.float64)
    again = out.clone()
    got = dca.embed_backward(grad, ids, V, scale=scale, accumulate=accumulate, out=out)
    assert got is out
    dca.embed_backward(grad, ids, V, scale=scale, accumulate=accumulate, out=again)
    torch.cuda.synchronize()
    total, size, count = plain.embed_backward(host(grad), ids.cpu().numpy(), V, float(np.float32(scale)))
    steps = np.minimum(count, np.maximum(256, 64 + count // 256 + 17))[:, None]
    bound = size * (steps + 2) * H * 1.01
    if accumulate:
        bound = bound + np.where(count[:, None] > 0, np.abs(was) + size, 0.0) * H
        total = total + was
    bound = bound + (np.abs(total) + bound) * np.where(count[:, None] > 0, HALF[otype], 0.0) + 2.0 ** -140
    assert (np.abs(host(out) - total) <= bound).all(), label
    assert torch.equal(out.view(torch.int16 if otype is BF16 else torch.int32) if out.is_contiguous() else out,
                       again.view(torch.int16 if otype is BF16 else torch.int32) if out.is_contiguous() else again)
    untouched = count == 0
    if accumulate:
        assert np.array_equal(host(out)[untouched], was[untouched])
    else:
        assert not host(out)[untouched].any()


@pytest.mark.parametrize("gtype,otype", [(F32, F32), (F32, BF16), (BF16, F32), (BF16, BF16)])
@pytest.mark.parametrize("n,V,d,pad,shift", [
    (1, 1, 1, 0, 0), (2, 5, 3, 1, 1), (16, 64, 64, 0, 0), (33, 1000, 130, 0, 3), (256, 70, 1030, 1, 1),
    (257, 70, 20, 1, 1), (200, 3000, 2, 0, 0), (50, 7, 9001, 0, 0), (1025, 77, 5, 3, 1),
    (700, 3001, 1029, 0, 1), (4097, 40000, 12, 0, 0)])
def test_embed_backward(n, V, d, pad, shift, gtype, otype):
    for kind in ("even", "one", "few", "outside", "none", "zipf"):
        grad, ids = matrix(n, d, gtype, n + d, pad, shift), tokens(n, V, kind, n)
        check_backward(grad, ids, V, 0.7, otype, False, pad, shift, kind)
        check_backward(grad, ids, V, 0.7, otype, True, pad, shift, kind)


@pytest.mark.parametrize("n,V,kind", [(8192, 200000, "zipf"), (8193, 1000, "even"), (20000, 63, "even"),
                                      (20001, 300000, "zipf"), (16385, 5, "one"), (30000, 64, "outside"),
                                      (70000, 4097, "few")])
def test_embed_backward_of_many_tokens(n, V, kind):
    """Both sorts, and both tiles."""
    grad, ids = matrix(n, 6, F32, 3), tokens(n, V, kind, 9)
    check_backward(grad, ids, V, 1.0, F32)
    check_backward(grad, ids, V, 1.0, F32, True)


def test_rows_of_blocks_and_strides():
    wide = matrix(12, 40, F32, 2).view(4, 3, 40)
    grad, ids = wide[:, :2, 3:20], tokens(8, 30, "zipf", 4).view(4, 2)
    want = dca.embed_backward(grad.reshape(8, 17).contiguous(), ids.view(-1), 30)
    assert torch.equal(dca.embed_backward(grad, ids, 30), want)
    assert torch.equal(dca.embed_backward(grad.transpose(0, 1), ids.t().contiguous(), 30, dtype=BF16).float(),
                       dca.embed_backward(grad.transpose(0, 1).contiguous(), ids.t().contiguous(), 30, dtype=BF16).float())
    one = matrix(1, 17, F32, 8).view(1, 1, 17).expand(4, 2, 17)  # one row for all
    assert torch.equal(dca.embed_backward(one, ids, 30), dca.embed_backward(one.contiguous(), ids, 30))
    out = torch.zeros((4, 3, 40), device="cuda")
    dca.embed(wide.view(12, 40), ids, out=out[:, 1:])
    assert torch.equal(out[:, 1:], dca.embed(wide.view(12, 40), ids)) and not out[:, 0].any()


def test_no_tokens():
    table = matrix(5, 4, F32, 1)
    none = torch.empty((0,), dtype=torch.int32, device="cuda")
    assert dca.embed(table, none).shape == (0, 4)
    assert dca.embed(table, none.view(2, 0)).shape == (2, 0, 4)
    grad = torch.empty((0, 4), device="cuda")
    out = table.clone()
    assert torch.equal(dca.embed_backward(grad, none, 5, accumulate=True, out=out), table)
    assert not dca.embed_backward(grad, none, 5, out=out).any()
    assert not dca.embed_backward(grad.view(2, 0, 4), none.view(2, 0), 5).any()


def test_infinities_stay_in_their_rows():
    grad = torch.ones((40, 5), device="cuda")
    grad[3, 2], grad[7, 1] = float("nan"), float("inf")
    ids = (torch.arange(40, device="cuda") % 20).int()
    ids[9] = -1
    grad[9] = float("nan")
    out = host(dca.embed_backward(grad, ids, 20))
    assert np.isnan(out[3, 2]) and out[7, 1] == np.inf
    out[3, 2] = out[7, 1] = 2.0
    want = np.full((20, 5), 2.0)
    want[9] = 1.0
    assert np.array_equal(out, want)


def test_gradient_against_differences():
    """The product of the gradient with a direction is the difference of the looked-up rows' along it (linear in the
    table, so exactly but for roundings)."""
    table, step = matrix(11, 9, F32, 1).double().cpu(), matrix(11, 9, F32, 2).double().cpu()
    ids, g = tokens(50, 11, "even", 3), matrix(50, 9, F32, 4)
    got = dca.embed_backward(g, ids, 11, scale=1.5).double().cpu()
    look = lambda t: dca.embed(t.float().cuda(), ids, scale=1.5).double().cpu()  # noqa: E731
    change = ((look(table + step) - look(table - step)) * g.double().cpu()).sum() / 2
    size = (got.abs() * step.abs()).sum() + (look(table.abs() + step.abs()) * g.double().cpu().abs()).sum()
    assert abs((got * step).sum() - change) <= 100 * H * size


def test_captured_twice_on_one_workspace_and_another_stream():
    V, d = 500, 33
    grads, ids = [matrix(300, d, F32, s) for s in (1, 2)], [tokens(300, V, "zipf", s) for s in (1, 2)]
    want = [dca.embed_backward(g, i, V) for g, i in zip(grads, ids)]
    ws = torch.empty(dca.embed_backward_workspace_size(300, 1, d), dtype=torch.uint8, device="cuda")
    outs = [torch.full((V, d), 7.0, device="cuda") for _ in range(2)]
    stream, graphs = torch.cuda.Stream(), []
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        dca.embed_backward(grads[0], ids[0], V, workspace=ws, out=outs[0])
    torch.cuda.current_stream().wait_stream(stream)
    assert torch.equal(outs[0], want[0])
    for k in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[k]):
            dca.embed_backward(grads[k], ids[k], V, workspace=ws, out=outs[k])
    for _ in range(4):
        for k in (1, 0):
            outs[k].fill_(3.0)
            graphs[k].replay()
        torch.cuda.synchronize()
        for k in range(2):
            assert torch.equal(outs[k], want[k])
        outs[0].sum().item()


def test_refusals_on_the_device():
    table, ids = matrix(5, 4, F32, 1), tokens(3, 5, "even", 1)
    with pytest.raises(ValueError, match="requires a gradient"):
        dca.embed(table.clone().requires_grad_(), ids)
    for bad in (ids.long(), ids.cpu(), ids.float(), torch.stack([ids, ids], 1)[:, 0]):
        with pytest.raises(ValueError):
            dca.embed(table, bad)
    with pytest.raises(dca.DominoError, match="overlap"):
        dca.embed(table, ids, out=table[:3])
    with pytest.raises(dca.DominoError, match="overlap"):
        dca.embed_backward(table[:3], ids, 5, out=table)
    with pytest.raises(dca.DominoError, match="overlap"):
        dca.embed_backward(table[:3], ids, 5, out=torch.zeros((1, 4), device="cuda").expand(5, 4))
    with pytest.raises(dca.DominoError, match="EWORKSPACE"):
        dca.embed_backward(matrix(300, 4, F32, 1), tokens(300, 5, "even", 1), 5,
                           workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(dca.DominoError):
        dca.embed(table, ids, scale=float("nan"))
    with pytest.raises(ValueError):
        dca.embed_backward(table[:3], ids, 5, accumulate=True)
    with pytest.raises(ValueError):
        dca.embed_backward(table[:3], ids, 5, out=torch.empty((4, 4), device="cuda"))
    with pytest.raises(ValueError):
        dca.embed_backward(table, ids, 5)
