"""Training a Markov head on tokens: embedding, linear layers and token log-probabilities together, as `adapt` runs
them."""
import numpy as np
import pytest
import torch

import causal_draft_correction_amd as dca
import domino_synth as ds
from causal_draft_correction_amd import adapt
from gpu_common import LF_TOL

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dca.load_library()


def small(B, V=3001, K=6):
    sh = ds.HeadShape(d=256, h=64, r=32, V=V, K=K, wdtype="bf16")
    w = dca.head_weights_to_device(ds.make_weights(sh, (31, 0), gru_sensitive=True))
    inp = ds.make_inputs(sh, B, (31, 1), sigma=0.5, peak="none")
    args = [dca.device_tensor(x) for x in (inp.H, inp.L_base, inp.last_tok)]
    g = torch.Generator().manual_seed(B)
    return w, args, torch.randint(0, V, (B, K), generator=g).int().cuda()


def parameters(w):
    return [torch.nn.Parameter(t) for t in (w["W1"].float(), w["W2"].float(), adapt.markov_table(w))]


def test_the_table_and_the_logits_are_the_markov_heads():
    w, (H, L, last), tokens = small(5)
    head = dca.DominoHead(w, K=6, max_batch=5, markov=True)
    want = head.draft(H, L, last, teacher=tokens, want_logits=True)["L_final"]
    W1, W2, table = parameters(w)
    with torch.no_grad():
        prev = torch.cat([last[:, None], tokens[:, :-1]], 1).contiguous()
        u = dca.linear(torch.cat([H.float(), dca.embed(table, prev)], -1), W1, activation="silu")["y"]
        got = dca.linear(u, W2, residual=L)["y"]
    assert (got - want).abs().max() <= LF_TOL


@pytest.mark.parametrize("lengths", [None, [6, 0, 3]])
@pytest.mark.parametrize("entropy", [0.0, 0.1])
def test_gradients_against_autograd_in_64_bits(lengths, entropy):
    w, (H, L, last), tokens = small(3)
    tokens[0, 4] = -1
    tokens[2, 1] = tokens[0, 0]  # rows of the table that several positions share
    params = parameters(w)
    n_rows = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    got = adapt.token_step(*params, H, L, last, tokens, n_rows=n_rows, entropy=entropy)
    # the same in float64 on the host
    W1, W2, T = (p.detach().double().cpu().requires_grad_() for p in params)
    t, h = tokens.long().cpu(), H.double().cpu()
    prev = torch.cat([last.long().cpu()[:, None], t[:, :-1]], 1)
    S = T[prev.clamp(min=0)] * (prev >= 0)[..., None]
    u = torch.nn.functional.silu(torch.cat([h, S], -1) @ W1.t())
    logp = torch.log_softmax(L.double().cpu() + u @ W2.t(), -1)
    counts = t >= 0
    if lengths is not None:
        counts &= torch.arange(t.shape[1]) < torch.tensor(lengths)[:, None]
    each = logp.gather(2, t.clamp(min=0)[..., None])[..., 0] + entropy * torch.special.entr(logp.exp()).sum(-1)
    loss = -(each * counts).sum() / counts.sum()
    loss.backward()
    # float32 sums of at most 3001 terms, through four products: 1e-5 of the largest gradient is far above their errors
    # (3001 half steps of the sum of magnitudes) and far below what a missing term would leave
    assert abs(float(got["loss"]) - float(loss)) <= 1e-5 * abs(float(loss))
    for p, q in zip(params, (W1, W2, T)):
        off = (p.grad.double().cpu() - q.grad).abs().max()
        assert off <= 1e-5 * q.grad.abs().max() * 10 and float(q.grad.abs().max()) > 0
    assert not got["logprob"][0, 4] and torch.isfinite(got["logprob"]).all()


def test_the_example_trains_on_tokens(capsys):
    got = adapt.main(steps=2)
    assert "on tokens: mean log-probability" in capsys.readouterr().out
    assert np.isfinite(got["token_losses"]).all() and len(got["token_losses"]) == 2
