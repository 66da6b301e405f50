"""The token step's gradients element by element, each against what float32 may leave of its own terms, with positions
that do not count inside the rows.

Bounds, H = 2^-24: errors are carried through the step's formulas on magnitudes, to first order in H (times 1.01 for what
is beyond).  A product of n float32 terms, here below the 320 from which on sums are cut into parts: 6 n additions of a step
(2 H) at most, H for the planes left out, of the sum of magnitudes.  silu and its slope: 24 H and 4 |a| H of themselves; the slopes of silu and of
its slope are at most 1.1 and 0.5.  Probabilities: a row's logits off by at most e move p by 2 e p and log p by 2 e, their
own evaluation by 40 H of p and of 1 + |log p|."""
import pytest
import torch

import causal_draft_correction_amd as dca
import domino_synth as ds
from causal_draft_correction_amd import adapt
from test_gpu_token_step import parameters, small

pytestmark = pytest.mark.gpu

H = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dca.load_library()


def few(B, V=300, K=6):
    """A head with sums of fewer than 320 terms, and logits far apart, so that entropies differ."""
    sh = ds.HeadShape(d=192, h=64, r=32, V=V, K=K, wdtype="bf16")
    w = dca.head_weights_to_device(ds.make_weights(sh, (33, 0), gru_sensitive=True))
    inp = ds.make_inputs(sh, B, (33, 1), sigma=0.5, peak="none")
    h, L, last = (dca.device_tensor(x) for x in (inp.H, inp.L_base, inp.last_tok))
    g = torch.Generator().manual_seed(B)
    return w, (h, 3 * L / L.std(), last), torch.randint(0, V, (B, K), generator=g).int().cuda()


def off(n, size):
    assert n < 320
    return (12 * n + 1) * H * size


def forms(W1, W2, T, h, L, t, prev, counts, entropy):
    """Loss, gradients of W1, W2 and the table, and the errors they may have."""
    d, V = h.shape[-1], W2.shape[0]
    h, L, t, prev, counts = (z.reshape((-1,) + z.shape[2:]) for z in (h, L, t, prev, counts))
    known = (prev >= 0) & (prev < V)
    S = T[prev.clamp(0, V - 1)] * known[:, None]
    x = torch.cat([h, S], 1)
    a, e_a = x @ W1.t(), off(x.shape[1], x.abs() @ W1.abs().t())
    s = torch.sigmoid(a)
    u = a * s
    e_u = 1.1 * e_a + u.abs() * (24 + 4 * a.abs()) * H
    l = L + u @ W2.t()
    e_l = e_u @ W2.abs().t() + off(u.shape[1], u.abs() @ W2.abs().t()) + (l.abs() + L.abs()) * 2 * H
    logp = torch.log_softmax(l, 1)
    p, ent = logp.exp(), torch.special.entr(logp.exp()).sum(1, keepdim=True)
    e = 2 * e_l.max(1, keepdim=True).values + 40 * H
    w = (counts.double() / counts.sum())[:, None]
    hit = torch.nn.functional.one_hot(t.clamp(min=0), V)
    G = w * (p - hit + entropy * p * (logp + ent))
    e_G = w * p * e * (1 + entropy * (logp.abs() + ent + 4)) + w * (1 - p) * hit * 8 * H + G.abs() * 8 * H
    loss = -(w * ((logp * hit).sum(1, keepdim=True) + entropy * ent)).sum()
    dW2 = G.t() @ u
    e_W2 = e_G.t() @ u.abs() + G.abs().t() @ e_u + off(len(x), G.abs().t() @ u.abs())
    U = G @ W2
    e_U = e_G @ W2.abs() + off(V, G.abs() @ W2.abs())
    slope = s * (1 + a * (1 - s))
    dp = U * slope
    e_dp = e_U * slope.abs() + U.abs() * (0.5 * e_a + s * (1 + a.abs() * (1 - s)) * (24 + 4 * a.abs()) * H) + dp.abs() * 2 * H
    dW1, e_W1 = dp.t() @ x, e_dp.t() @ x.abs() + off(len(x), dp.abs().t() @ x.abs())
    dS, e_dS = dp @ W1[:, d:], e_dp @ W1[:, d:].abs() + off(len(W1), dp.abs() @ W1[:, d:].abs())
    dT, e_T = torch.zeros_like(T), torch.zeros_like(T)
    dT.index_add_(0, prev[known], dS[known])
    e_T.index_add_(0, prev[known], e_dS[known] + len(x) * 2 * H * dS[known].abs())
    return loss, [(dW1, e_W1), (dW2, e_W2), (dT, e_T)]


@pytest.mark.parametrize("lengths", [None, [6, 0, 3]])
@pytest.mark.parametrize("entropy", [0.0, 0.1])
@pytest.mark.parametrize("given", [False, True])
def test_each_element(lengths, entropy, given):
    w, (h, L, last), tokens = few(3)
    whole = tokens.clone()  # what the rows hold
    tokens[0, 4] = tokens[1, 0] = tokens[2, 2] = -1
    whole[2, 1] = whole[0, 0]
    tokens[2, 1] = tokens[0, 0]
    previous = torch.cat([last[:, None], whole[:, :-1]], 1).contiguous()
    params = parameters(w)
    n_rows = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    got = adapt.token_step(*params, h, L, last, tokens, n_rows=n_rows, entropy=entropy,
                           previous=previous if given else None)
    counts = tokens.cpu() >= 0
    if lengths is not None:
        counts &= torch.arange(6) < torch.tensor(lengths)[:, None]
    prev = previous if given else torch.cat([last[:, None], tokens[:, :-1]], 1)
    loss, wants = forms(*(q.detach().double().cpu() for q in params), h.double().cpu(), L.double().cpu(),
                        tokens.long().cpu(), prev.long().cpu(), counts, entropy)
    assert abs(float(got["loss"].detach()) - float(loss)) <= 1e-5 * abs(float(loss))
    for q, (want, bound) in zip(params, wants):
        assert ((q.grad.double().cpu() - want).abs() <= 1.01 * bound + 2.0 ** -120).all()
        live = want.abs().sum(1) > 0
        assert float(q.grad[~live.cuda()].abs().sum()) == 0
    if given:  # a state of the table for every position: the rows that precede counted positions, and no others
        rows = set(previous.cpu()[counts].tolist())
        assert set(params[2].grad.abs().sum(1).nonzero()[:, 0].tolist()) == rows


@pytest.mark.parametrize("left_out", ["entropy", "a position", "state"])
def test_the_bounds_show_what_is_left_out(left_out):
    """The formulas with a term less, against themselves: each gradient goes out of its bounds, and where the term is in
    many rows, in a good part of them."""
    g = torch.Generator().manual_seed(5)

    def normal(*shape):
        return torch.randn(shape, generator=g, dtype=torch.float64)

    W1, W2, T = normal(32, 256) / 16, normal(300, 32) / 6, normal(300, 64) / 2
    h, L = normal(3, 6, 192), 3 * normal(3, 6, 300)
    t = torch.randint(0, 300, (3, 6), generator=g)
    prev = torch.randperm(300, generator=g)[:18].view(3, 6)
    counts = torch.ones((3, 6), dtype=torch.bool)
    _, right = forms(W1, W2, T, h, L, t, prev, counts, 0.1)
    other = {"entropy": counts, "state": counts, "a position": counts.clone()}[left_out]
    if left_out == "a position":
        other[1, 3] = False
    before = torch.where(torch.arange(18).view(3, 6) == 7, -1, prev) if left_out == "state" else prev
    _, wrong = forms(W1, W2, T, h, L, t, before, other, 0.0 if left_out == "entropy" else 0.1)
    for (want, bound), (got, _) in zip(right, wrong):
        seen = ((got - want).abs() > 1.01 * bound).any(1)
        touched = (got - want).abs().sum(1) > 0
        assert seen.any() and (left_out == "state" or seen[touched].double().mean() > 0.4)


def test_the_tokens_before_are_the_default():
    w, (h, L, last), tokens = small(2)
    params, again = parameters(w), parameters(w)
    adapt.token_step(*params, h, L, last, tokens)
    adapt.token_step(*again, h, L, last, tokens, previous=torch.cat([last[:, None], tokens[:, :-1]], 1).contiguous())
    assert all(torch.equal(p.grad, q.grad) for p, q in zip(params, again))
    for bad in (last[:, None], tokens.long(), tokens[:, :5].contiguous()):
        with pytest.raises(ValueError):
            adapt.token_step(*params, h, L, last, tokens, previous=bad)
