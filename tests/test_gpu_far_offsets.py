"""Operands whose elements lie more than 2^32 apart: layers and token log-probabilities on rows of one large buffer,
against the same calls on the rows next to each other.  The buffer's other memory is not touched (and not initialised)."""
import pytest
import torch

import causal_draft_correction_amd as dca

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
STEP = 2 ** 31 + 40  # elements from a row to the next


@pytest.fixture(scope="module")
def buffer():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dca.load_library()
    return torch.empty(3 * STEP + 4096, dtype=BF16, device="cuda")  # 12.9 GB


def far(buffer, rows, cols, seed=None, dtype=BF16):
    """[rows, cols] with STEP elements (of dtype) from row to row."""
    t = buffer.view(dtype).as_strided((rows, cols), (STEP * BF16.itemsize // dtype.itemsize, 1)) if dtype is F32 else \
        buffer.as_strided((rows, cols), (STEP, 1))
    if seed is not None:
        g = torch.Generator(device="cuda").manual_seed(seed)
        t.copy_(torch.randn((rows, cols), generator=g, device="cuda"))
    return t


def test_linear(buffer):
    x = far(buffer, 3, 70, 1)
    w, near = torch.randn((90, 70), device="cuda"), x.contiguous()
    want = dca.linear(near, w, dtype=F32)["y"]
    assert torch.equal(dca.linear(x, w, dtype=F32)["y"], want)
    # as weights, as residual, as output
    y = torch.randn((20, 70), device="cuda").to(BF16)
    assert torch.equal(dca.linear(y, x, dtype=F32)["y"], dca.linear(y, near, dtype=F32)["y"])
    g = torch.randn((20, 3), device="cuda")
    a, b = (dca.linear_backward(g, y, t) for t in (x, near))
    assert torch.equal(a["x"], b["x"]) and torch.equal(a["weight"], b["weight"])
    out = far(buffer, 3, 90, 2)
    want = dca.linear(near, w, residual=out.contiguous(), dtype=BF16)["y"]
    dca.linear(near, w, residual=out, out={"y": out})
    assert torch.equal(out, want)
    grad = far(buffer, 3, 90, 3)
    flat = grad.contiguous()
    a, b = (dca.linear_backward(t, near, w, want=("x", "weight", "bias")) for t in (grad, flat))
    assert all(torch.equal(a[n], b[n]) for n in a)


def test_embedding(buffer):
    d = 1000
    V = buffer.numel() // d
    table = buffer[:V * d].view(V, d)  # 6.4 million rows: the last begins past 2^32 elements
    ids = torch.tensor([V - 1, 0, V - 2, V, V - 1, V // 2], dtype=torch.int32, device="cuda")
    for v in (0, V // 2, V - 2, V - 1):
        table[v] = torch.randn(d, device="cuda")
    got = dca.embed(table, ids, scale=2.0)
    want = table[ids.long().clamp(max=V - 1)] * 2
    want[3] = 0
    assert torch.equal(got, want)
    rows = far(buffer, 3, d, 5)
    three = torch.tensor([1, 4, 1], dtype=torch.int32, device="cuda")
    assert torch.equal(dca.embed_backward(rows, three, 6), dca.embed_backward(rows.contiguous(), three, 6))
    many = torch.full((300,), V - 1, dtype=torch.int32, device="cuda")
    grad = torch.randn((300, d), device="cuda")
    table[V - 1] = 0
    dca.embed_backward(grad, many, V, accumulate=True, out=table)
    assert torch.equal(table[V - 1], dca.embed_backward(grad, torch.zeros_like(many), 1, dtype=BF16)[0])


@pytest.mark.parametrize("V", [3000, 70001])
def test_token_logprobs(buffer, V):
    if V > 4000:
        z = buffer.as_strided((2, V), (STEP, 1))
        z.copy_(torch.randn((2, V), device="cuda"))
    else:
        z = far(buffer, 3, V, 1)
    near = z.contiguous()
    n = z.shape[0]
    tokens = torch.arange(n, device="cuda").int() * 7
    g = torch.ones(n, device="cuda")
    for kw in (dict(), dict(k=5)):
        a, b = dca.token_logprobs(z, tokens, **kw), dca.token_logprobs(near, tokens, **kw)
        assert all(torch.equal(a[name], b[name]) for name in a)
    want = dca.token_logprobs(near, tokens, grad_logprob=g, grad_entropy=g)["grad"]
    assert torch.equal(dca.token_logprobs(z, tokens, grad_logprob=g, grad_entropy=g, out={"grad": z})["grad"], want)
    assert torch.equal(z, want)
