"""GPU results of linear layers and their gradients against their plain 64-bit forms (layers_plain.py).

Bounds, in halves of a float32 step (H = 2^-24).  A sum of n products takes n additions for each product of two parts
of the operands (1 for bfloat16, 3 for a float32 one, 6 for two), and one for each part of the sum that is joined; each
is off by at most a step (2 H, were it cut instead of rounded) of the sum of magnitudes.  The parts of two float32
operands that are not multiplied weigh at most 2^-26 = H / 4.  The activations: an exponential or erfc of its own (16 H
at most together with the divisions and products around it), whose argument is off by 2 H of itself, which moves
erfc(a / sqrt 2) by 2 a^2 H and exp(a) by 2 |a| H of itself.  Their slopes do not exceed 1.2, so an error of pre counts
1.2 times.  Then the output's type."""
import numpy as np
import pytest
import torch

import causal_draft_correction_amd as dca
import layers_plain as plain
from test_gpu_embed import BF16, F32, H, HALF, host, matrix

pytestmark = pytest.mark.gpu

TINY = 2.0 ** -120
TYPES = [(F32, F32), (F32, BF16), (BF16, F32), (BF16, BF16)]
SHAPES = [(1, 1, 1), (3, 7, 5), (2, 33, 300), (16, 256, 1000), (17, 40, 130), (16, 64, 64), (129, 65, 131),
          (331, 1091, 203), (128, 512, 128), (200, 2000, 64), (5, 5120, 256), (257, 300, 1031), (1000, 16, 33),
          (64, 4097, 70)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dca.load_library()


def f64(t):
    return host(t).astype(np.float64)


def parts(*types):
    n = sum(t is F32 for t in types)
    return (1, 3, 6)[n]


def sum_bound(n, size, *types):
    return (parts(*types) * n + 600) * 2 * H * size + H / 4 * size + TINY


def act_error(a, name):
    """Of act(a), for a itself."""
    size = np.abs(plain.act(a, name))
    return {"silu": size * (16 + 2 * np.abs(a)) * H, "gelu": size * (16 + 2 * a * a) * H, "relu": 0.0 * a,
            None: 0.0 * a}[name] + TINY


def slope_error(a, name):
    if name == "silu":
        with np.errstate(over="ignore"):
            s, o = 1 / (1 + np.exp(-a)), 1 / (1 + np.exp(a))
        return s * (1 + np.abs(a) * o) * (24 + 4 * np.abs(a)) * H + TINY
    if name == "gelu":
        return (plain.slope(-np.abs(a), name).__abs__() + np.abs(a) * np.exp(-0.5 * a * a) + (a > 0)) * \
            (24 + 4 * a * a) * H + TINY
    return 0.0 * a


def check(got, want, bound, label):
    got = f64(got) if isinstance(got, torch.Tensor) else got
    bad = np.abs(got - want) > bound
    assert not bad.any(), "%s: %d of %d, worst %g of its bound" % (label, bad.sum(), bad.size,
                                                                  (np.abs(got - want) / bound).max())


def rounded(want, bound, dtype):
    return bound + (np.abs(want) + bound) * HALF[dtype] + TINY


def same_bits(a, b):
    return a.dtype is b.dtype and torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


class Guarded:
    """A tensor in a buffer whose other elements have to stay as they are."""

    def __init__(self, rows, cols, dtype, pad, shift, seed=77):
        self.t = matrix(rows, cols, dtype, seed, pad, shift)
        n = self.t.untyped_storage().nbytes() // self.t.element_size()
        self.all = torch.as_strided(self.t, (n,), (1,), 0)
        self.was = self.all.clone()

    def kept(self):
        mask = torch.ones_like(self.all, dtype=torch.bool)
        torch.as_strided(mask, self.t.shape, self.t.stride(), self.t.storage_offset()).fill_(False)
        return same_bits(self.all[mask], self.was[mask])


@pytest.mark.parametrize("xt,wt", TYPES)
@pytest.mark.parametrize("M,K,N", SHAPES)
def test_linear(M, K, N, xt, wt):
    seed = M + K + N
    x, w = matrix(M, K, xt, seed, 3, 1), matrix(N, K, wt, seed + 1, 0, 0)
    want, size = plain.product(host(x), host(w))
    got = dca.linear(x, w, dtype=F32)["y"]
    check(got, want, rounded(want, sum_bound(K, size, xt, wt), F32), "product")
    assert same_bits(got, dca.linear(x, w, dtype=F32)["y"])
    # everything at once, into padded rows
    for act, yt, rt, bt in (("silu", BF16, F32, BF16), ("gelu", F32, BF16, F32), ("relu", F32, F32, F32)):
        bias, residual = matrix(1, N, bt, 5)[0], matrix(M, N, rt, 6, 1, 1)
        y, pre = Guarded(M, N, yt, 2, 3), Guarded(M, N, F32, 1, 0)
        dca.linear(x, w, bias=bias, activation=act, residual=residual, out={"y": y.t, "pre": pre.t})
        a = want + host(bias)
        e = sum_bound(K, size, xt, wt) + (np.abs(a) + size) * 2 * H
        check(pre.t, a, rounded(a, e, F32), act + " pre")
        full = plain.act(a, act) + host(residual)
        e = 1.2 * e + act_error(a, act) + (np.abs(full) + np.abs(host(residual))) * 2 * H
        check(y.t, full, rounded(full, e, yt), act)
        assert y.kept() and pre.kept()


# Sizes of each kind of tile, with edges that fill none: 512 x 256 results over a long sum; 256 tiles of 256 x 256 and
# more (bfloat16), and the same sizes with a float32 operand.
LONG = [("y", 300, 263, 20003), ("x", 300, 261, 20003), ("weight", 517, 262, 20003), ("y", 261, 20003, 300),
        ("y", 4100, 523, 4098), ("x", 4100, 4098, 523), ("weight", 523, 4098, 4100)]


@pytest.mark.parametrize("at,bt", TYPES)
@pytest.mark.parametrize("kind,M,K,N", LONG)
def test_long_products(kind, M, K, N, at, bt):
    """Against float64 products on the device (numpy's would take a minute)."""
    if kind == "y":
        a, b = matrix(M, K, at, 1, 1, 1), matrix(N, K, bt, 2)
        want, n = lambda x, y: x @ y.t(), K  # noqa: E731
        residual, bias = matrix(M, N, F32, 3), matrix(1, N, F32, 4)[0]
        got = dca.linear(a, b, bias=bias, activation="relu", residual=residual, want_pre=True)
        pre = want(a.double(), b.double()) + bias.double()
        size = want(a.double().abs(), b.double().abs()) + bias.abs()
        bound = (parts(at, bt) * n + 600) * 2 * H * size + H / 4 * size + pre.abs() * H + TINY
        assert ((got["pre"].double() - pre).abs() <= bound).all()
        y = pre.clamp(min=0) + residual.double()
        assert ((got["y"].double() - y).abs() <= bound + (y.abs() + residual.abs()) * 2 * H).all()
        return
    g = matrix(M, N, at, 1, 0, 1)
    other = matrix(N, K, bt, 2) if kind == "x" else matrix(M, K, bt, 2)
    x, w = (matrix(M, K, bt, 5), other) if kind == "x" else (other, matrix(N, K, bt, 5))
    want, n = ((lambda p, q: p @ q), N) if kind == "x" else ((lambda p, q: p.t() @ q), M)
    out = matrix(M, K, F32, 9, 3, 1) if kind == "x" else matrix(N, K, F32, 9, 3, 1)
    dca.linear_backward(g, x, w, want=(kind,), out={kind: out})
    size = want(g.double().abs(), other.double().abs())
    bound = (parts(at, bt) * n + 600) * 2 * H * size + H / 4 * size + TINY
    assert ((out.double() - want(g.double(), other.double())).abs() <= bound).all()


def test_linear_without_rounding():
    """Operands whose products and sums float32 holds: every bit of the result."""
    g = torch.Generator().manual_seed(3)
    for M, K, N in ((5, 37, 70), (130, 64, 140), (40, 700, 65), (300, 200, 20003), (2100, 515, 8200)):
        x = torch.randint(-2 ** 5, 2 ** 5, (M, K), generator=g)
        w = torch.randint(-2 ** 5, 2 ** 5, (N, K), generator=g)
        want = (x.double() @ w.double().t()).float()
        for xt, wt in TYPES:
            assert torch.equal(dca.linear(x.to(xt).cuda(), w.to(wt).cuda(), dtype=F32)["y"].cpu(), want)
    # one product each, of 24 bits: x = 1 + 2^-23, w a power of two, and all of x's bits one by one
    x = torch.cat([1 + 2.0 ** -torch.arange(1, 24).float(), -(2.0 ** torch.arange(-60, 60, 7).float()) * (1 + 2.0 ** -23)])
    w = torch.tensor([[1.0], [-2.0 ** 20], [2.0 ** -30]])
    for wt in (F32, BF16):
        got = dca.linear(x.view(-1, 1).cuda(), w.to(wt).cuda())["y"].cpu()
        assert torch.equal(got, x.view(-1, 1) * w.t())


def test_small_products_keep_24_bits():
    """float32 operands with few terms: no more than the parts left out and the additions' own rounding."""
    for K in (1, 2, 8):
        x, w = matrix(70, K, F32, K), matrix(150, K, F32, K + 1)
        want, size = plain.product(host(x), host(w))
        # (6 K additions of a step at most: the bound without the allowance for joins)
        check(dca.linear(x, w)["y"], want, (6 * K + 1) * 2 * H * size, "K=%d" % K)


@pytest.mark.parametrize("gt,wt", TYPES)
@pytest.mark.parametrize("M,K,N", SHAPES)
def test_linear_backward(M, K, N, gt, wt):
    seed = M + K + N
    xt = wt if (M + K) % 2 else (F32 if wt is BF16 else BF16)
    g, x, w = matrix(M, N, gt, seed, 1, 1), matrix(M, K, xt, seed + 1, 0, 1), matrix(N, K, wt, seed + 2, 5, 0)
    for act in (None, "silu", "gelu", "relu"):
        pre = None if act is None else matrix(M, N, F32, 8, 1, 0).mul_(3)
        dpre, e, dt = f64(g), 0.0 * f64(g), gt
        if act:
            a = f64(pre)
            e = np.abs(dpre) * (slope_error(a, act) + np.abs(plain.slope(a, act)) * 2 * H)
            dpre, dt = dpre * plain.slope(a, act), F32
        dx, dw, db = Guarded(M, K, BF16 if act else F32, 2, 1), Guarded(N, K, F32 if act else BF16, 0, 0), \
            Guarded(1, N, F32, 0, 0)
        was_w, was_b = f64(dw.t), f64(db.t)
        out = {"x": dx.t, "weight": dw.t, "bias": db.t[0]}
        got = dca.linear_backward(g, x, w, pre=pre, activation=act, want=("x", "weight", "bias"), out=out)
        assert got["x"] is dx.t
        wants = {}
        want, size = plain.product(dpre, host(w).T)
        wants["x"] = want, sum_bound(N, size, dt, wt) + 1.01 * plain.product(e, host(w).T)[1]
        want, size = plain.product(dpre.T, host(x).T)
        wants["weight"] = want, sum_bound(M, size, dt, xt) + 1.01 * plain.product(e.T, host(x).T)[1]
        want, size = dpre.sum(0)[None], np.abs(dpre).sum(0)[None]
        wants["bias"] = want, (M + 70) * 2 * H * size + 1.01 * e.sum(0)[None] + TINY
        for name, t in (("x", dx.t), ("weight", dw.t), ("bias", db.t)):
            check(t, wants[name][0], rounded(*wants[name], t.dtype), "%s of %s" % (name, act))
        assert dx.kept() and dw.kept()
        # each alone, twice: the same bits
        for name in out:
            one = dca.linear_backward(g, x, w, pre=pre, activation=act, want=(name,),
                                      out={name: torch.empty_like(out[name])})
            assert set(one) == {name} and same_bits(one[name], out[name])
        # added to what is there
        dw.all.copy_(dw.was), db.all.copy_(db.was)
        dca.linear_backward(g, x, w, pre=pre, activation=act, want=("weight", "bias"), accumulate=True,
                            out={"weight": dw.t, "bias": db.t[0]})
        for name, t, was in (("weight", dw.t, was_w), ("bias", db.t, was_b)):
            want, bound = wants[name][0] + was, wants[name][1] + (np.abs(was) + np.abs(wants[name][0])) * 2 * H
            check(t, want, rounded(want, bound, t.dtype), "%s added" % name)


@pytest.mark.parametrize("act", [None, "silu", "gelu", "relu"])
def test_gradients_against_differences(act):
    """Directional derivatives from the forward pass itself, central differences of its float32 results."""
    M, K, N, step = 37, 50, 41, 2.0 ** -7
    x, w, b, g = (matrix(*s, F32, i) for i, s in enumerate([(M, K), (N, K), (1, N), (M, N)]))
    b = b[0]
    pre = dca.linear(x, w, bias=b, want_pre=True)["pre"]
    got = dca.linear_backward(g, x, w, pre=None if act is None else pre, activation=act, want=("x", "weight", "bias"))
    for name, t, i in (("x", x, 0), ("weight", w, 1), ("bias", b, 2)):
        d = matrix(*(t.shape if t.dim() == 2 else (1, N)), F32, 20 + i).view(t.shape)

        def value(s):
            args = [x, w, b]
            args[i] = t + s * d
            p = dca.linear(args[0], args[1], bias=args[2], want_pre=True)["pre"]
            if act == "relu":  # (its slope by the sides the values are on, without the kink between)
                y = torch.where(pre > 0, p, torch.zeros_like(p))
                return f64(y), (f64(y) * f64(g)).sum()
            y = dca.linear(args[0], args[1], bias=args[2], activation=act)["y"]
            return f64(y), (f64(y) * f64(g)).sum()

        (y1, v1), (y0, v0) = value(step), value(-step)
        slope = (v1 - v0) / (2 * step)
        # the results' own errors over the step, and the third derivative (below 2 for these activations)
        _, size = plain.product(host(x), host(w))
        noise = (np.abs(f64(g)) * (sum_bound(K, 2 * size + 4, F32, F32) * 1.2 + (np.abs(y1) + 1) * 40 * H)).sum() / step
        moved = {"x": plain.product(host(d).reshape(-1, d.shape[-1]), host(w))[1] if i == 0 else None,
                 "weight": plain.product(host(x), host(d))[1] if i == 1 else None,
                 "bias": np.broadcast_to(np.abs(host(d)), (M, N)) if i == 2 else None}[name]
        third = 0.0 if act in (None, "relu") else (np.abs(f64(g)) * moved ** 3).sum() * 2 * step ** 2 / 6
        mine = (f64(got[name]) * f64(d)).sum()
        assert abs(mine - slope) <= noise + third + 1e-4 * abs(slope), name


def test_blocks_of_rows_and_strides():
    wide = matrix(40, 60, F32, 2).view(8, 5, 60)
    x, w = wide[:, :3, 7:40], matrix(21, 33, BF16, 3, 9, 2)
    flat = x.reshape(24, 33).contiguous()
    for xx, ff in ((x, flat), (x.transpose(0, 1), x.transpose(0, 1).reshape(24, 33).contiguous()),
                   (x[:, :1].expand(8, 3, 33), x[:, :1].expand(8, 3, 33).reshape(24, 33).contiguous())):
        lead = xx.shape[:2]
        want = dca.linear(ff, w, activation="silu", want_pre=True)
        got = dca.linear(xx, w, activation="silu", want_pre=True)
        assert got["y"].shape == lead + (21,)
        assert same_bits(got["y"].view(24, 21), want["y"]) and same_bits(got["pre"].view(24, 21), want["pre"])
        g = matrix(lead[0] * 4, 21, F32, 5).view(lead[0], 4, 21)[:, 1:4] if lead[1] == 3 else \
            matrix(24, 21, F32, 5).view(3, 8, 21)
        a = dca.linear_backward(g, xx, w, pre=got["pre"], activation="silu", want=("x", "weight", "bias"))
        b = dca.linear_backward(g.reshape(24, 21).contiguous(), ff, w, pre=want["pre"], activation="silu",
                                want=("x", "weight", "bias"))
        assert same_bits(a["x"].view(24, 33), b["x"]) and same_bits(a["weight"], b["weight"]) and \
            same_bits(a["bias"], b["bias"])
    # part of a weight matrix, columns of it
    both = matrix(21, 90, F32, 9)
    assert same_bits(dca.linear(flat, both[:, 50:83])["y"], dca.linear(flat, both[:, 50:83].contiguous())["y"])


def test_the_residual_in_place_and_masked_logits():
    x, w = matrix(20, 64, F32, 1), matrix(3001, 64, BF16, 2)
    base = matrix(20, 3001, F32, 3)
    base[:, 5::7] = -np.inf
    base[3] = torch.finfo(F32).min
    want = dca.linear(x, w, residual=base)["y"]
    y = base.clone()
    got = dca.linear(x, w, residual=y, out={"y": y})["y"]
    assert got is y and same_bits(y, want)
    assert (y[:, 5::7] == -np.inf)[[0, 1, 2, 4]].all() and torch.isfinite(y[3, 0])
    with pytest.raises(dca.DominoError, match="overlap"):
        dca.linear(x, w, residual=y, out={"y": torch.as_strided(y, (20, 3001), (2800, 1), 1)})


def test_infinities_and_nan_stay_in_their_rows():
    for xt, wt in TYPES:
        x, w = matrix(30, 40, xt, 1), matrix(50, 40, wt, 2)
        clean = host(dca.linear(x, w, dtype=F32)["y"])
        x[4, 7], x[9, 0] = float("nan"), float("inf")
        w[11, 3] = float("-inf")
        got = host(dca.linear(x, w, dtype=F32)["y"])
        assert not np.isfinite(got[4]).any() and not np.isfinite(got[9]).any() and not np.isfinite(got[:, 11]).any()
        keep = np.ix_([i for i in range(30) if i not in (4, 9)], [i for i in range(50) if i != 11])
        assert np.array_equal(got[keep], clean[keep])
    pre = torch.tensor([[-3e38, -200.0, -90.0, -0.0, 0.0, 90.0, 200.0, 3e38]], device="cuda")
    one = torch.ones((1, 1), device="cuda")
    for act, slopes in (("silu", [0, 0, 0, 0.5, 0.5, 1, 1, 1]), ("gelu", [0, 0, 0, 0.5, 0.5, 1, 1, 1]),
                        ("relu", [0, 0, 0, 0, 0, 1, 1, 1])):
        y = host(dca.linear(one, torch.zeros((8, 1), device="cuda"), bias=pre[0], activation=act)["y"])[0]
        # (silu(-90) = -90 e^-90)
        assert np.allclose(y, [0, 0, 0, 0, 0, 90, 200, np.float32(3e38)], rtol=1e-6, atol=1e-36)
        got = dca.linear_backward(torch.ones((1, 8), device="cuda"), one, torch.zeros((8, 1), device="cuda"), pre=pre,
                                  activation=act, want=("bias",))["bias"]
        assert np.allclose(host(got), slopes, rtol=1e-6, atol=1e-36)


def test_no_rows():
    w = matrix(6, 5, F32, 1)
    for x, g in ((torch.empty((0, 5), device="cuda"), torch.empty((0, 6), device="cuda")),
                 (torch.empty((2, 0, 5), device="cuda"), torch.empty((2, 0, 6), device="cuda"))):
        got = dca.linear(x, w, activation="silu", want_pre=True)
        assert got["y"].shape == got["pre"].shape == g.shape
        out = dca.linear_backward(g, x, w, pre=got["pre"], activation="silu", want=("x", "weight", "bias"))
        assert out["x"].shape == x.shape and not out["weight"].any() and not out["bias"].any()
        assert out["weight"].shape == (6, 5)
        was = {"weight": w.clone(), "bias": w[:, 0].contiguous()}
        out = dca.linear_backward(g, x, w, want=("weight", "bias"), accumulate=True,
                                  out={n: t.clone() for n, t in was.items()})
        assert torch.equal(out["weight"], was["weight"]) and torch.equal(out["bias"], was["bias"])


def test_captured_twice_on_one_workspace_and_another_stream():
    M, K, N = 40, 2000, 70
    x, w, g = matrix(M, K, F32, 1), matrix(N, K, BF16, 2), matrix(M, N, F32, 3)
    pre = dca.linear(x, w, want_pre=True)["pre"]
    kw = dict(pre=pre, activation="silu", want=("x", "weight", "bias"))
    want_y, want = dca.linear(x, w, activation="silu")["y"], dca.linear_backward(g, x, w, **kw)
    need = max(dca.linear_workspace_size(M, 1, K, N, "silu", (F32, BF16)),
               dca.linear_backward_workspace_size(M, 1, K, N, "silu", kw["want"], (F32, F32, BF16)))
    assert dca.linear_workspace_size(M, 1, K, N, None, (F32, BF16)) > 0  # (its sums are shared out)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        y = dca.linear(x, w, activation="silu", workspace=ws)["y"]
        got = dca.linear_backward(g, x, w, workspace=ws, **kw)
    torch.cuda.current_stream().wait_stream(stream)
    assert same_bits(y, want_y) and all(same_bits(got[n], want[n]) for n in want)
    y = torch.empty_like(want_y)
    out = {n: torch.empty_like(t) for n, t in want.items()}
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    with torch.cuda.graph(graphs[0]):
        dca.linear(x, w, activation="silu", workspace=ws, out={"y": y})
    with torch.cuda.graph(graphs[1]):
        dca.linear_backward(g, x, w, workspace=ws, out=out, **kw)
    for _ in range(4):
        y.fill_(3.0)
        for t in out.values():
            t.fill_(3.0)
        graphs[1].replay()
        graphs[0].replay()
        torch.cuda.synchronize()
        assert same_bits(y, want_y) and all(same_bits(out[n], want[n]) for n in want)
        x.sum().item()


def test_refusals_on_the_device():
    x, w, g = matrix(4, 8, F32, 1), matrix(6, 8, F32, 2), matrix(4, 6, F32, 3)
    for call in (lambda: dca.linear(x, w.clone().requires_grad_()), lambda: dca.linear(x, w, activation="tanh"),
                 lambda: dca.linear(x, w[:, :7]), lambda: dca.linear(x, w, bias=x[0]), lambda: dca.linear(x, w, residual=x),
                 lambda: dca.linear(x, w.double()), lambda: dca.linear(x, w, out={"z": g}),
                 lambda: dca.linear(x, w.t().contiguous().t()), lambda: dca.linear_backward(g, x, w, want=()),
                 lambda: dca.linear_backward(g, x, w, want=("y",)), lambda: dca.linear_backward(g, x, w[:5]),
                 lambda: dca.linear_backward(g, x, w, accumulate=True),
                 lambda: dca.linear_backward(g, x, w, out={"weight": x}), lambda: dca.linear(x.cpu(), w)):
        with pytest.raises((ValueError, dca.DominoError)):
            call()
    for call in (lambda: dca.linear(x, w, out={"y": torch.as_strided(x, (4, 6), (8, 1))}),
                 lambda: dca.linear_backward(g, x, w, out={"weight": w}),
                 lambda: dca.linear_backward(g, x, w, pre=g), lambda: dca.linear_backward(g, x, w, activation="relu"),
                 lambda: dca.linear(x, w, out={"y": torch.zeros((1, 6), device="cuda").expand(4, 6)})):
        with pytest.raises(dca.DominoError):
            call()
    need = dca.linear_workspace_size(4, 1, 5000, 6, None, (BF16, BF16))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")  # as much as it says is enough, and no less
    exact = matrix(4, 5000, BF16, 1), matrix(6, 5000, BF16, 2)
    dca.linear(*exact, workspace=ws)
    with pytest.raises(dca.DominoError, match="EWORKSPACE"):
        dca.linear(*exact, workspace=ws[:-1])
    wide = matrix(4, 5000, F32, 1), matrix(6, 5000, F32, 2)
    with pytest.raises(dca.DominoError, match="EWORKSPACE"):
        dca.linear(*wide, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_long_rows_of_blocks_that_lie_apart(dtype):
    wide, w = matrix(40 * 5, 230, dtype, 1).view(40, 5, 230), matrix(130, 200, dtype, 2)
    for x in (wide[:, 1:4, 9:209], wide[:, 1:4, 9:209].transpose(0, 1), wide[:, :1, 3:203].expand(40, 3, 200)):
        g = wide[:, 1:4, 50:180] if x.shape[0] == 40 else wide[:, 1:4, 50:180].transpose(0, 1)
        assert same_bits(dca.linear(x, w)["y"], dca.linear(x.contiguous(), w)["y"])
        got, want = dca.linear_backward(g, x, w), dca.linear_backward(g.contiguous(), x.contiguous(), w)
        assert same_bits(got["x"], want["x"]) and same_bits(got["weight"], want["weight"])
