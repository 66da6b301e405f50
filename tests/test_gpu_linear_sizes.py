"""Linear layers whose result is wide one way and narrow the other, and around the sizes where one kind of tile gives way
to the next, against float64 products on the device.  Whole numbers below 2^5, so that float32 has every sum: every bit."""
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


def whole(rows, cols, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-2 ** 5, 2 ** 5, (rows, cols), generator=g, device="cuda").to(dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M", [16, 17, 64, 127, 128, 129, 192])
def test_few_rows_onto_a_vocabulary(M, dtype):
    K, N = 520, 65573
    x, w, g = whole(M, K, dtype, M), whole(N, K, dtype, 1), whole(M, N, dtype, 2)
    want = x.double() @ w.double().t()
    assert torch.equal(dca.linear(x, w, dtype=F32)["y"].double(), want)
    # (about 2^16 terms below 2^10: those of one sign add up to less than 2^24, so float32 has the sum of any of them)
    want, size = g.double() @ w.double(), g.double().abs() @ w.double().abs()
    assert (size + want.abs()).max() / 2 < 2 ** 24
    got = dca.linear_backward(g, x, w, want=("x",), out={"x": torch.empty((M, K), device="cuda")})["x"]
    assert torch.equal(got.double(), want)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("K", [1, 3, 16, 64, 128, 129, 256])
@pytest.mark.parametrize("M", [511, 512])
def test_gradient_of_narrow_weights(M, K, dtype):
    N = 65573
    x, w, g = whole(M, K, dtype, K), whole(N, K, dtype, 1), whole(M, N, dtype, 2)
    was = whole(N, K, F32, 3)
    for accumulate in (False, True):
        out = was.clone()
        dca.linear_backward(g, x, w, want=("weight",), accumulate=accumulate, out={"weight": out})
        want = g.double().t() @ x.double() + (was.double() if accumulate else 0)
        assert torch.equal(out.double(), want)
