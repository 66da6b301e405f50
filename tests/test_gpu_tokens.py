"""GPU results of token log-probabilities against their plain 64-bit form (tokens_plain.py, which derives the bounds)."""
import numpy as np
import pytest
import torch

import causal_draft_correction_amd as dca
import rows_plain
import tokens_plain as plain
from test_gpu_rows import special_rows

pytestmark = pytest.mark.gpu

H = plain.H
F32, BF16 = torch.float32, torch.bfloat16
HALF = {F32: H, BF16: 2.0 ** -8}
DTYPES = [F32, BF16]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dca.load_library()


def rows(B, R, V, dtype, seed, pad=0, shift=0, scale=3.0):
    """[B, R, V] logits, a view of a buffer with `pad` columns after each row and `shift` elements before the first."""
    g = torch.Generator().manual_seed(seed)
    flat = torch.randn(shift + B * R * (V + pad), generator=g).mul_(scale).to(dtype).cuda()
    return flat[shift:].view(B, R, V + pad)[..., :V]


def host(t):
    return t.float().cpu().numpy()


def bits(t):
    return t.contiguous().view(torch.uint8).cpu()


def near(got, want, bound, label):
    assert np.array_equal(np.isnan(got), np.isnan(want)), label
    with np.errstate(over="ignore"):  # (a log-probability below float32's lowest is -inf there)
        inf = np.isinf(want.astype(np.float32))
        want = np.where(inf, want.astype(np.float32), want)
    assert np.array_equal(got[inf], want[inf]), label
    ok = np.isfinite(want)
    over = np.where(ok, np.abs(np.where(ok, got, 0) - np.where(ok, want, 0)) - bound, -1.0)
    at = np.unravel_index(np.argmax(over), over.shape)
    assert over[at] <= 0, "%s: %r instead of %r +- %r at %s" % (label, got[at], want[at], bound[at], at)


def check(z, tokens, k=0, tau=1.0, n_rows=None, label="", grads=True):
    """Every form of the call: with and without alternatives and statistics, the gradient by itself, together, in place."""
    B, R, V = z.shape
    nr = None if n_rows is None else torch.tensor(n_rows, dtype=torch.int32, device="cuda")
    tok = torch.as_tensor(tokens, dtype=torch.int32).reshape(B, R).contiguous().cuda()
    t, zh = tok.cpu().numpy(), host(z)
    kw = dict(temperature=tau, n_rows=nr)
    ref = [[plain.row(zh[b, r], int(t[b, r]) if n_rows is None or r < n_rows[b] else -1, tau) for r in range(R)]
           for b in range(B)]
    pick = lambda name: np.array([[x[name] for x in line] for line in ref])  # noqa: E731
    calls = [dca.token_logprobs(z, tok, want_stats=True, **kw), dca.token_logprobs(z, tok, **kw)]
    if k:
        calls += [dca.token_logprobs(z, tok, k=k, want_stats=True, **kw), dca.token_logprobs(z, tok, k=k, **kw)]
    for got in calls:
        near(host(got["logprob"]), pick("logprob"), pick("logprob_err"), label + " logprob")
        near(host(got["entropy"]), pick("entropy"), pick("entropy_err"), label + " entropy")
    for a, b in zip(calls[::2], calls[1::2]):
        assert all(torch.equal(bits(a[n]), bits(b[n])) for n in b), label
    if k:
        ids = rows_plain.top(zh, k, 1.0, n_rows)[0]
        live = pick("live") | (pick("logprob") == -np.inf)
        ids[~live] = -1
        assert np.array_equal(calls[2]["ids"].cpu().numpy(), ids), label
        want = np.full((B, R, k), -np.inf)
        bound = np.zeros((B, R, k))
        for b in range(B):
            for r in range(R):
                if live[b, r]:
                    want[b, r] = ref[b][r]["logp"][ids[b, r]]
                    bound[b, r] = ref[b][r]["rel"] + np.abs(np.nan_to_num(want[b, r], posinf=0, neginf=0)) * H + plain.TINY
        near(host(calls[2]["logprobs"]), want, bound, label + " alternatives")
    if not grads:
        return
    g = torch.Generator().manual_seed(5)
    g1, g2 = torch.randn((B, R), generator=g).cuda(), torch.randn((B, R), generator=g).cuda()
    for a, b in ((g1, g2), (g1, None), (None, g2)):
        ga, gb = (np.zeros((B, R)) if x is None else host(x).astype(np.float64) for x in (a, b))
        want, bound = np.zeros(z.shape), np.zeros(z.shape)
        for i in range(B):
            for r in range(R):
                want[i, r], bound[i, r] = plain.gradient(ref[i][r], int(t[i, r]), tau, ga[i, r], gb[i, r])
        bound = bound + (np.abs(want) + bound) * HALF[z.dtype] + (2.0 ** -133 if z.dtype is BF16 else 0)
        own = z.clone()
        outs = [dca.token_logprobs_backward(z, tok, c["stats"], a, b, **kw) for c in calls[::2]]
        both = dca.token_logprobs(z, tok, grad_logprob=a, grad_entropy=b, **kw)
        outs.append(both["grad"])
        near(host(both["logprob"]), pick("logprob"), pick("logprob_err"), label + " logprob")
        near(host(both["entropy"]), pick("entropy"), pick("entropy_err"), label + " entropy")
        outs.append(dca.token_logprobs(own, tok, grad_logprob=a, grad_entropy=b, out={"grad": own}, **kw)["grad"])
        assert outs[-1] is own and torch.equal(bits(own), bits(both["grad"]))
        outs.append(dca.token_logprobs_backward(z, tok, calls[0]["stats"], a, b, out=z.clone(), **kw))
        assert torch.equal(bits(outs[-1]), bits(outs[0]))
        for i, got in enumerate(outs):
            near(host(got), want, bound, "%s gradient %d" % (label, i))


def some_tokens(B, R, V, seed, z=None):
    g = torch.Generator().manual_seed(seed)
    t = torch.randint(0, V, (B, R), generator=g)
    if z is not None:  # every other one the likeliest
        t.view(-1)[::2] = z.float().reshape(B * R, V).argmax(1).cpu()[::2]
    return t


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,R,V,k,pad,shift,tau", [
    (1, 1, 1, 1, 0, 0, 1.0), (1, 3, 7, 7, 0, 1, 1.0), (2, 3, 130, 5, 3, 0, 0.5), (1, 2, 1024, 128, 0, 0, 1.0),
    (2, 1, 1025, 64, 0, 3, 2.0), (1, 1, 2048, 1, 5, 1, 1.0), (3, 2, 5003, 33, 0, 0, 0.1), (1, 1, 16384, 128, 0, 0, 1.0),
    (2, 2, 16385, 100, 7, 1, 0.7), (1, 2, 40001, 128, 0, 0, 10.0), (1, 1, 151936, 64, 0, 0, 1.0),
    (30, 40, 1099, 17, 1, 0, 1.0), (1, 2, 32769, 7, 0, 1, 1.0), (2, 1, 65537, 5, 3, 0, 1.0), (20, 14, 33001, 3, 1, 1, 1.0)])
def test_token_logprobs(B, R, V, k, pad, shift, tau, dtype):
    z = rows(B, R, V, dtype, 7 * V + k, pad, shift)
    check(z, some_tokens(B, R, V, 3, z), k, tau, label="V=%d" % V)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V,k", [(300, 100), (2100, 9), (30001, 60), (70000, 128)])
def test_special_rows(V, k, dtype):
    named = special_rows(V, dtype)
    z = torch.stack(list(named.values())).cuda().view(1, len(named), V)
    for seed in (1, 2):
        tokens = some_tokens(1, len(named), V, seed, z if seed == 1 else None)
        check(z, tokens, k, 1.0, label="special")
        check(z, tokens, 0, 1e-4, label="cold")
    check(z, tokens, 0, 1e4, label="hot")


@pytest.mark.parametrize("dtype", DTYPES)
def test_rows_that_are_nearly_certain(dtype):
    """What is left of the others shows in all digits: in the log-probability, the entropy and both gradients."""
    for V in (513, 9000, 40000):
        z = rows(1, 8, V, dtype, V, scale=1.0)
        at = torch.arange(8) * 37 + 5
        for r in range(8):
            z[0, r, at[r]] = z.float().max().item() + 2.0 ** r
        tokens = at.clone()
        tokens[3] = 1
        check(z, tokens, 3, label="certain")
        got = dca.token_logprobs(z, tokens.view(1, 8).int().cuda())
        assert (got["logprob"][0, [0, 1, 2, 4, 5]] < 0).all()  # exp(-32) of it still shows


def test_shifted_rows():
    """A row far from 0 keeps its differences, on both sides of where the exponent's form changes."""
    z = rows(1, 3, 3000, F32, 4)
    for by in (50.0, 500.0, 1000.0, 1e4, -1e4):
        moved = (z.double() + by).float()  # (rounded: the logits are what they are then)
        check(moved, some_tokens(1, 3, 3000, 2, moved), 5, label="by %g" % by)


def test_lengths_ignored_tokens_strides_and_two_dimensions():
    wide = rows(4, 6, 3001, F32, 5)
    tokens = some_tokens(4, 5, 3001, 1)
    tokens[0, 3], tokens[2, 0], tokens[3, 1], tokens[3, 4] = -1, 3001, -100, 2 ** 31 - 1
    check(wide[:, :5], tokens, 9, 1.0, [0, 1, 5, 99], "slice of rows")
    check(wide[:, :5], tokens, 9, 1.0, None, "ignored tokens")
    check(wide[:, 1:2].expand(4, 5, 3001), tokens, 4, 2.0, None, "one row for all")
    check(wide[:, :5].transpose(0, 1), tokens.t(), 4, 1.0, None, "batch and rows exchanged")
    check(wide[:1, :5], tokens[:1], 0, 1.0, [-3], "negative length")
    two = dca.token_logprobs(wide[0], tokens.new_tensor([1, 2, 3, 4, 5, 6]).int().cuda(), k=3)
    three = dca.token_logprobs(wide[:1], tokens.new_tensor([[1, 2, 3, 4, 5, 6]]).int().cuda(), k=3)
    assert all(torch.equal(two[n], three[n][0]) for n in two)
    long = rows(3, 2, 50000, BF16, 8, 3, 1)
    check(long, [[1, -1], [5, 49999], [50000, 3]], 5, 1.0, [2, 2, 1], "chunks")
    none = torch.empty((0, 4, 50), device="cuda")
    got = dca.token_logprobs(none, torch.empty((0, 4), dtype=torch.int32, device="cuda"), k=2)
    assert got["ids"].shape == (0, 4, 2) and got["logprob"].shape == (0, 4)


def test_results_do_not_depend_on_left_out_rows_memory():
    z = rows(2, 3, 700, F32, 1)
    z[0, 2] = float("nan")
    z[1, 1] = float("inf")
    tokens = torch.tensor([[1, 2, 3], [4, -1, 6]], dtype=torch.int32, device="cuda")
    g = torch.ones((2, 3), device="cuda")
    got = dca.token_logprobs(z, tokens, grad_logprob=g, grad_entropy=g,
                             n_rows=torch.tensor([2, 3], dtype=torch.int32, device="cuda"))
    for r in ((0, 2), (1, 1)):
        assert got["logprob"][r] == 0 and got["entropy"][r] == 0 and not got["grad"][r].any()
    assert torch.isfinite(got["grad"]).all()


@pytest.mark.parametrize("tau", [0.5, 1.0, 3.0])
def test_gradient_against_differences(tau):
    """Central differences of the call's own results along random directions."""
    V, step = 400, 2.0 ** -6
    z, d = rows(1, 6, V, F32, 3), rows(1, 6, V, F32, 4, scale=1.0)
    tokens = some_tokens(1, 6, V, 2, z).int().cuda()
    g1, g2 = torch.randn((1, 6), device="cuda"), torch.randn((1, 6), device="cuda")
    got = dca.token_logprobs(z, tokens, temperature=tau, grad_logprob=g1, grad_entropy=g2)

    def value(s):
        out = dca.token_logprobs((z.double() + s * step * d.double()).float(), tokens, temperature=tau)
        return out["logprob"].double() * g1 + out["entropy"].double() * g2

    slope = (value(1) - value(-1)) / (2 * step)
    mine = (got["grad"].double() * d.double()).sum(-1)
    # third derivatives of both are below 100 (moments of d, at most 5, over tau); the results' errors below 2^-18, and
    # the rounding of z moves them by its own half steps
    bound = (g1.abs() + g2.abs()).double() * (100 / tau ** 3 * step ** 2 / 6 + (2.0 ** -18 + 16 * H / tau * 20) / step)
    assert ((slope - mine).abs() <= bound).all()


def test_workspace_streams_and_captured_graphs():
    B, R, V, k = 2, 5, 70001, 7
    z = [rows(B, R, V, BF16, s) for s in (1, 2)]
    tok = [some_tokens(B, R, V, s).int().cuda() for s in (1, 2)]
    g = torch.randn((B, R), device="cuda")
    want = [(dca.token_logprobs(a, t, k=k), dca.token_logprobs(a, t, grad_logprob=g, grad_entropy=g)) for a, t in zip(z, tok)]
    need = max(dca.token_logprobs_workspace_size(B, R, V, n, BF16) for n in (0, k))
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    outs = [({n: torch.empty_like(x) for n, x in w[0].items()}, {n: torch.empty_like(x) for n, x in w[1].items()})
            for w in want]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        dca.token_logprobs(z[0], tok[0], k=k, workspace=ws, out=outs[0][0])
    torch.cuda.current_stream().wait_stream(stream)
    assert all(torch.equal(outs[0][0][n], want[0][0][n]) for n in want[0][0])
    graphs = []
    for i in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            dca.token_logprobs(z[i], tok[i], k=k, workspace=ws, out=outs[i][0])
            dca.token_logprobs(z[i], tok[i], grad_logprob=g, grad_entropy=g, workspace=ws, out=outs[i][1])
    for _ in range(4):
        for i in (1, 0):
            for o in outs[i]:
                for x in o.values():
                    x.zero_()
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            for o, w in zip(outs[i], want[i]):
                assert all(torch.equal(o[n], w[n]) for n in w)
        g.sum().item()


def test_refusals_on_the_device():
    z, tok = rows(2, 3, 50, F32, 1), torch.zeros((2, 3), dtype=torch.int32, device="cuda")
    g = torch.ones((2, 3), device="cuda")
    stats = dca.token_logprobs(z, tok, want_stats=True)["stats"]
    for call in (lambda: dca.token_logprobs(z, tok.long()), lambda: dca.token_logprobs(z, tok[:, :2]),
                 lambda: dca.token_logprobs(z, tok.cpu()), lambda: dca.token_logprobs(z.requires_grad_(False).double(), tok),
                 lambda: dca.token_logprobs(z.clone().requires_grad_(), tok),
                 lambda: dca.token_logprobs(z, tok, k=2, grad_logprob=g), lambda: dca.token_logprobs(z, tok, out={"ids": tok}),
                 lambda: dca.token_logprobs(z, tok, want_stats=True, grad_entropy=g),
                 lambda: dca.token_logprobs(z, tok, grad_logprob=g[:1]),
                 lambda: dca.token_logprobs_backward(z, tok, stats), lambda: dca.token_logprobs_backward(z, tok, g, g),
                 lambda: dca.token_logprobs_backward(z, tok, stats, g, out=z.to(BF16))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: dca.token_logprobs(z, tok, k=-1), lambda: dca.token_logprobs(z, tok, k=129),
                 lambda: dca.token_logprobs(z, tok, k=51), lambda: dca.token_logprobs(z, tok, temperature=0.0),
                 lambda: dca.token_logprobs(z, tok, grad_logprob=g, out={"grad": torch.zeros((1, 1, 50), device="cuda").expand(2, 3, 50)}),
                 lambda: dca.token_logprobs(z, tok, out={"logprob": z.view(-1)[:6].view(2, 3)}),
                 lambda: dca.token_logprobs(rows(2, 3, 40000, F32, 1), tok,
                                            workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(dca.DominoError):
            call()
    with torch.no_grad():
        dca.token_logprobs(z.clone().requires_grad_(), tok)
