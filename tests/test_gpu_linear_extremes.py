"""Linear layers on infinities, NaN and the largest finite values, against what the definition's products and sums give:
an infinity times a number that is not 0 is infinite, times 0 it is NaN, infinities of both signs add up to NaN, and a
float32 that bfloat16 would round to infinity is a finite number like any other."""
import pytest
import torch

import causal_draft_correction_amd as dca

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
TYPES = [(F32, F32), (F32, BF16), (BF16, F32), (BF16, BF16)]
# kinds of tiles and ways to them: less than a step of the sum, whole steps and a rest, 16 rows, a sum in parts, 128 x 128
SHAPES = [(5, 7, 9), (70, 96, 130), (70, 101, 131), (16, 64, 300), (40, 2000, 70), (2051, 515, 2049)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dca.load_library()


def small_numbers(rows, cols, dtype, seed):
    """Whole numbers below 8, among them zeros: float32 has every sum of their products."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-7, 8, (rows, cols), generator=g, device="cuda").to(dtype)


def spoil(t, seed):
    """Infinities and NaN in a few places, a row with two infinities among them."""
    g = torch.Generator().manual_seed(seed)
    rows, cols = t.shape
    for value in (float("inf"), float("-inf"), float("inf"), float("nan")):
        t[int(torch.randint(rows, (1,), generator=g)), int(torch.randint(cols, (1,), generator=g))] = value
    t[rows // 2, 0], t[rows // 2, cols - 1] = float("inf"), float("-inf")
    return t


def product(x, w):
    """x w^T by what its terms are, in float64 without an infinity in a product."""
    x, w = x.double(), w.double()

    def count(a, b):
        return a.double() @ b.double().t() > 0

    every_x, every_w = torch.ones_like(x), torch.ones_like(w)
    nan = count(x.isnan(), every_w) | count(every_x, w.isnan()) | count(x.isinf(), w == 0) | count(x == 0, w.isinf())
    inf = float("inf")
    up = count(x == inf, w > 0) | count(x == -inf, w < 0) | count(x > 0, w == inf) | count(x < 0, w == -inf)
    down = count(x == inf, w < 0) | count(x == -inf, w > 0) | count(x > 0, w == -inf) | count(x < 0, w == inf)
    zero = torch.zeros((), dtype=torch.float64, device="cuda")
    y = torch.where(x.isfinite(), x, zero) @ torch.where(w.isfinite(), w, zero).t()
    y[up], y[down] = inf, -inf
    y[nan | (up & down)] = float("nan")
    return y


def same(got, want):
    got = got.double()
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got.nan_to_num(nan=0.5, posinf=1e300, neginf=-1e300),
                       want.nan_to_num(nan=0.5, posinf=1e300, neginf=-1e300))


@pytest.mark.parametrize("xt,wt", TYPES)
@pytest.mark.parametrize("M,K,N", SHAPES)
def test_products_with_infinities(M, K, N, xt, wt):
    for first, second in ((True, False), (False, True), (True, True)):
        x, w = small_numbers(M, K, xt, 1), small_numbers(N, K, wt, 2)
        if first:
            spoil(x, 3)
        if second:
            spoil(w, 4)
        same(dca.linear(x, w, dtype=F32)["y"], product(x, w))
        g = small_numbers(M, N, xt, 5)
        if first:
            spoil(g, 6)
        grads = {"x": torch.empty((M, K), device="cuda"), "weight": torch.empty((N, K), device="cuda")}
        dca.linear_backward(g, x, w, out=grads)
        same(grads["x"], product(g, w.t()))
        same(grads["weight"], product(g.t(), x.t()))


@pytest.mark.parametrize("wt", [F32, BF16])
@pytest.mark.parametrize("M,K,N", SHAPES)
def test_the_largest_finite_values(M, K, N, wt):
    """One term of a row at float32's largest magnitudes, its factors powers of two or 0: exact products."""
    big = torch.finfo(F32).max
    x = torch.zeros((M, K), device="cuda")
    at = torch.arange(M, device="cuda") % K
    values = torch.tensor([big, -big, big * (1 - 2.0 ** -23), -3.39e38, 3.395e38], device="cuda")
    rows = torch.arange(M, device="cuda")
    x[rows, at] = values[rows % 5]
    g = torch.Generator(device="cuda").manual_seed(7)
    w = torch.tensor([0.0, 1.0, -1.0, 0.5, -2.0 ** -90], device="cuda")[
        torch.randint(5, (N, K), generator=g, device="cuda")].to(wt)
    want = x[rows, at].double()[:, None] * w.double()[:, at].t()
    assert torch.equal(dca.linear(x, w)["y"].double(), want)
    # as grad, and as x beside it
    assert torch.equal(dca.linear_backward(x, torch.zeros((M, N), device="cuda"), w.t().contiguous(),
                                           want=("x",))["x"].double(), want)
    one = torch.zeros((M, N), device="cuda")
    one[:, 0] = 1
    got = dca.linear_backward(one, x, torch.zeros((N, K), device="cuda"), want=("weight",))["weight"]
    want = torch.zeros((N, K), dtype=torch.float64, device="cuda")
    if M <= K:  # (a column of x has one value)
        want[0] = x.double().sum(0)
        assert torch.equal(got.double(), want)


def test_sums_that_overflow():
    """Products past float32 whose parts overflow with both signs."""
    for K in (3, 64, 200):
        x = torch.full((20, K), 1e30, device="cuda") * (1 + 2.0 ** -9 - 2.0 ** -20)
        w = torch.full((30, K), 1e30, device="cuda") * (1 + 2.0 ** -9 - 2.0 ** -20)
        w[7] *= -1
        y = dca.linear(x, w)["y"]
        assert (y[:, 7] == -float("inf")).all()
        keep = [i for i in range(30) if i != 7]
        assert (y[:, keep] == float("inf")).all()


def test_infinities_through_the_epilogue():
    """Bias, relu and residual after a product that is infinite."""
    x, w = small_numbers(9, 40, F32, 1), small_numbers(12, 40, F32, 2).abs().add_(1)
    x[3, 5], x[4, 6] = float("inf"), float("-inf")
    residual, bias = small_numbers(9, 12, F32, 3), small_numbers(1, 12, F32, 4)[0]
    got = dca.linear(x, w, bias=bias, activation="relu", residual=residual, want_pre=True)
    same(got["pre"], product(x, w) + bias.double())
    same(got["y"], (product(x, w) + bias.double()).clamp(min=0) + residual.double())
