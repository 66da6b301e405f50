"""Gradients of a few tokens added to a table: the rows that the tokens name and no others, each with its tokens' gradients
in the order of their places."""
import pytest
import torch

import causal_draft_correction_amd as dca

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dca.load_library()


@pytest.mark.parametrize("gtype,ttype", [(F32, F32), (BF16, F32), (F32, BF16), (BF16, BF16)])
@pytest.mark.parametrize("n,V,d", [(1, 1, 1), (1, 151936, 64), (32, 20011, 4096), (200, 77, 1031), (256, 5, 2049),
                                   (256, 100003, 100), (256, 1, 33)])
def test_rows_of_few_tokens(n, V, d, gtype, ttype):
    g = torch.Generator(device="cuda").manual_seed(n + d)
    ids = torch.randint(-1, V + 1, (n,), generator=g, device="cuda").int()
    ids[0], ids[-1] = V - 1, V - 1  # (first and last place the same token)
    grad = torch.randn((n, d + 3), generator=g, device="cuda").to(gtype)[:, 1:d + 1]
    table = torch.randn((V, d + 5), generator=g, device="cuda").to(ttype)
    was = table.clone()
    got = dca.embed_backward(grad, ids, V, scale=-0.5, accumulate=True, out=table[:, 2:d + 2])
    assert got.data_ptr() == table[:, 2:].data_ptr()
    # in float32, place after place, then the scale, the addition and the type
    want, sums = was.clone(), torch.zeros((V, d), device="cuda")
    for i, v in enumerate(ids.tolist()):
        if 0 <= v < V:
            sums[v] += grad[i].float()
    rows = ids[(ids >= 0) & (ids < V)].unique().long()
    want[rows, 2:d + 2] = (was[rows, 2:d + 2].double() - 0.5 * sums[rows].double()).to(F32).to(ttype)
    assert torch.equal(table, want)
    # onto zeros: the bits of the gradient that is not added
    zero = torch.zeros((V, d), device="cuda")
    assert torch.equal(dca.embed_backward(grad, ids, V, scale=3.0, accumulate=True, out=zero),
                       dca.embed_backward(grad, ids, V, scale=3.0, dtype=F32))


def test_no_token_of_the_table():
    table = torch.randn((50, 2000), device="cuda")
    was = table.clone()
    ids = torch.tensor([-1, 50, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device="cuda")
    dca.embed_backward(torch.randn((4, 2000), device="cuda"), ids, 50, accumulate=True, out=table)
    assert torch.equal(table, was)


def test_a_captured_addition():
    ids = torch.tensor([3, 9, 3, -1, 0], dtype=torch.int32, device="cuda")
    grad, table = torch.ones((5, 1500), device="cuda"), torch.zeros((10, 1500), device="cuda")
    dca.embed_backward(grad, ids, 10, accumulate=True, out=table)
    once = table.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dca.embed_backward(grad, ids, 10, accumulate=True, out=table)
    for times in range(2, 5):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(table, times * once)
