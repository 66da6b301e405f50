"""Linear layers: types of pre and of the bias' gradient, gradients added to what is there in every kind of tile, all bits
of float32 operands in every kind of tile, and rows as far apart as the 32-bit offsets of a tile reach.

Bounds as in test_gpu_linear.py.  A float32 operand's three planes multiply to all but H = 2^-24 of a product; with only two
planes of it up to 2^-17 would be missing."""
import numpy as np
import pytest
import torch

import causal_draft_correction_amd as dca
import layers_plain as plain
from test_gpu_embed import BF16, F32, H, HALF, host, matrix
from test_gpu_linear import Guarded, act_error, check, f64, rounded, same_bits, slope_error, sum_bound

pytestmark = pytest.mark.gpu

TYPES = [(F32, F32), (F32, BF16), (BF16, F32), (BF16, BF16)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dca.load_library()


@pytest.mark.parametrize("xt,wt", TYPES)
@pytest.mark.parametrize("M,K,N", [(3, 7, 5), (16, 256, 1000), (129, 65, 131), (5, 5120, 256), (257, 300, 1031)])
def test_pre_in_bfloat16(M, K, N, xt, wt):
    x, w, bias = matrix(M, K, xt, 1), matrix(N, K, wt, 2), matrix(1, N, F32, 3)[0]
    want, size = plain.product(host(x), host(w))
    a = want + host(bias)
    e = sum_bound(K, size, xt, wt) + (np.abs(a) + size) * 2 * H
    for act in (None, "silu", "gelu", "relu"):
        pre = Guarded(M, N, BF16, 3, 1)
        y = dca.linear(x, w, bias=bias, activation=act, dtype=F32, out={"pre": pre.t})["y"]
        check(pre.t, a, rounded(a, e, BF16), "pre")
        assert pre.kept()
        # (y is of the sums, not of what pre rounds them to)
        assert same_bits(y, dca.linear(x, w, bias=bias, activation=act, dtype=F32)["y"])
        check(y, plain.act(a, act), rounded(plain.act(a, act), 1.2 * e + act_error(a, act), F32), str(act))


@pytest.mark.parametrize("gt", [F32, BF16])
@pytest.mark.parametrize("pt", [F32, BF16])
@pytest.mark.parametrize("bt", [F32, BF16])
@pytest.mark.parametrize("M,K,N", [(1, 1, 1), (7, 5, 3), (40, 64, 203), (331, 40, 130), (1100, 9, 70)])
def test_bias_gradients(M, K, N, gt, pt, bt):
    g, x, w = matrix(M, N, gt, 1, 1, 1), matrix(M, K, F32, 2), matrix(N, K, F32, 3)
    for act in ("silu", "gelu", "relu"):
        pre = matrix(M, N, pt, 4, 2, 1).mul_(2)
        a = f64(pre)
        dpre = f64(g) * plain.slope(a, act)
        e = np.abs(f64(g)) * (slope_error(a, act) + np.abs(plain.slope(a, act)) * 2 * H)
        want, size = dpre.sum(0)[None], np.abs(dpre).sum(0)[None]
        bound = (M + 70) * 2 * H * size + 1.01 * e.sum(0)[None] + 2.0 ** -120
        out = matrix(1, N, bt, 5)
        was = f64(out)
        got = dca.linear_backward(g, x, w, pre=pre, activation=act, want=("bias",), out={"bias": torch.empty_like(out[0])})
        check(got["bias"][None], want, rounded(want, bound, bt), act)
        dca.linear_backward(g, x, w, pre=pre, activation=act, want=("bias",), accumulate=True, out={"bias": out[0]})
        check(out, want + was, rounded(want + was, bound + (np.abs(want) + np.abs(was)) * 2 * H, bt), act + " added")


# (M, K, N): both products in one launch, its sums in one part and in several; tiles of 128; tiles of 256 (bfloat16), its
# weight gradient wide and long
ADDED = [(64, 70, 50), (331, 1091, 203), (40, 2000, 70), (515, 2049, 2051), (523, 4098, 4100)]


@pytest.mark.parametrize("gt,xt", TYPES)
@pytest.mark.parametrize("wt", [F32, BF16])
@pytest.mark.parametrize("M,K,N", ADDED)
def test_all_gradients_added(M, K, N, gt, xt, wt):
    """Whole numbers below 2^4: float32 has every sum, in any order, and every sum with what is there."""
    g = torch.Generator(device="cuda").manual_seed(M)

    def whole(rows, cols, dtype, pad=0):
        return torch.randint(-2 ** 4, 2 ** 4, (rows, cols + pad), generator=g, device="cuda").to(dtype)[:, pad:]

    grad, x, w = whole(M, N, gt), whole(M, K, xt, 1), whole(N, K, F32)
    buffer, dx = whole(N, K, wt, 3), torch.empty((M, K), device="cuda")
    db = whole(1, N, wt)[0]
    was_w, was_b = buffer.clone(), db.clone()
    dca.linear_backward(grad, x, w, want=("x", "weight", "bias"), accumulate=True,
                        out={"x": dx, "weight": buffer, "bias": db})
    assert torch.equal(dx.double(), grad.double() @ w.double())
    # (one rounding, of the sum with what was there)
    assert torch.equal(buffer, (grad.double().t() @ x.double() + was_w.double()).float().to(wt))
    assert torch.equal(db, (grad.double().sum(0) + was_b.double()).float().to(wt))


# kinds of tiles (64 x 16, 64 x 64, 128 x 128) with whole steps of the sum
@pytest.mark.parametrize("M,K,N", [(16, 64, 300), (70, 96, 130), (2051, 544, 2049)])
@pytest.mark.parametrize("at,bt", TYPES[:3])
def test_all_bits_of_float32_operands(M, K, N, at, bt):
    """One term a row, of 24 random bits: 6 additions of a step (2 H) and the planes left out (H) of the product, each."""
    g = torch.Generator(device="cuda").manual_seed(K)

    def sparse(rows, cols, dtype):
        t = torch.zeros((rows, cols), device="cuda")
        at_row = torch.arange(rows, device="cuda")
        t[at_row, (at_row * 7) % cols] = torch.randn(rows, generator=g, device="cuda")
        return t.to(dtype)

    def dense(rows, cols, dtype):
        return torch.randn((rows, cols), generator=g, device="cuda").to(dtype)

    def near(got, a, b):
        want = a.double() @ b.double()
        off = (got.double() - want).abs()
        assert (off <= 13 * H * want.abs() + 2.0 ** -120).all(), float((off / want.abs().clamp(min=1e-30)).max() / H)

    x, w = sparse(M, K, at), dense(N, K, bt)
    near(dca.linear(x, w, dtype=F32)["y"], x, w.t())
    grad, w = sparse(M, N, at), dense(N, K, bt)
    near(dca.linear_backward(grad, x, w, want=("x",), out={"x": torch.empty((M, K), device="cuda")})["x"], grad, w)
    grad, x = dense(M, N, at), sparse(K, M, bt).t().contiguous()
    near(dca.linear_backward(grad, x, w, want=("weight",), out={"weight": torch.empty((N, K), device="cuda")})["weight"],
         grad.t(), x)
    # both gradients in one launch, where that is what their sizes take
    grad = sparse(M, N, at)
    x = sparse(K, M, bt).t().contiguous()
    out = {"x": torch.empty((M, K), device="cuda"), "weight": torch.empty((N, K), device="cuda")}
    dca.linear_backward(grad, x, w, out=out)
    near(out["x"], grad, w)
    near(out["weight"], grad.t(), x)


def planes(x, n):
    """x as float64 sums of its first n bfloat16 planes."""
    total, rest = torch.zeros_like(x, dtype=torch.float64), x.clone()
    for _ in range(n):
        part = rest.to(BF16).float()
        total += part.double()
        rest = rest - part
    return total


def test_that_bound_shows_a_missing_plane():
    """The same bound on the host: three planes are all of a float32, two leave more than it for most."""
    x = torch.randn(10000, generator=torch.Generator().manual_seed(1))
    assert torch.equal(planes(x, 3), x.double())
    assert ((planes(x, 2) - x.double()).abs() > 13 * H * x.double().abs()).double().mean() > 0.5


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rows_as_far_apart_as_offsets_reach(dtype):
    """Rows 2^21 - 1 elements apart are the farthest that a tile takes by 32-bit offsets; beside them 2^21, and blocks of
    rows that span just below and above 2^29 elements."""
    step, rows = 2 ** 21, 130
    buffer = torch.empty(step * rows + 4096, dtype=dtype, device="cuda")  # 1.1 GB in float32
    for stride in (step - 1, step):
        far = buffer.as_strided((rows, 200), (stride, 1))
        far.copy_(matrix(rows, 200, dtype, 1))
        close = far.contiguous()
        w, g = matrix(90, 200, dtype, 2), matrix(rows, 90, dtype, 3)
        assert same_bits(dca.linear(far, w)["y"], dca.linear(close, w)["y"])
        one, two = dca.linear_backward(g, far, w), dca.linear_backward(g, close, w)
        assert same_bits(one["x"], two["x"]) and same_bits(one["weight"], two["weight"])
        # as weights, and as grad: across the sum
        y, z = matrix(70, 200, dtype, 4), matrix(70, rows, dtype, 5)
        assert same_bits(dca.linear(y, far)["y"], dca.linear(y, close)["y"])
        assert same_bits(dca.linear_backward(z, y, far, want=("x",))["x"], dca.linear_backward(z, y, close, want=("x",))["x"])
        x = matrix(rows, 60, dtype, 6)
        v = matrix(200, 60, dtype, 7)
        one, two = dca.linear_backward(far, x, v, want=("x", "weight", "bias")), \
            dca.linear_backward(close, x, v, want=("x", "weight", "bias"))
        assert all(same_bits(one[n], two[n]) for n in one)
    del far, buffer
    B, R, K = 3, 33, 200
    buffer = torch.empty(2 ** 29 + 4096, dtype=dtype, device="cuda")
    for span in (2 ** 29 - 1, 2 ** 29):  # elements from the first to the one past the last
        bs = (span - K - (R - 1) * 1000) // (B - 1)
        rs = 1000
        far = buffer.as_strided((B, R, K), (bs, rs, 1), span - ((B - 1) * bs + (R - 1) * rs + K))
        far.copy_(matrix(B * R, K, dtype, 1).view(B, R, K))
        close, w = far.contiguous(), matrix(90, K, dtype, 2)
        assert same_bits(dca.linear(far, w)["y"], dca.linear(close, w)["y"])
        g = matrix(B * R, 90, dtype, 3).view(B, R, 90)
        one, two = dca.linear_backward(g, far, w), dca.linear_backward(g, close, w)
        assert same_bits(one["x"], two["x"]) and same_bits(one["weight"], two["weight"])
