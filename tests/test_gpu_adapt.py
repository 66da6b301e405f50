"""Beam drafts and distillation steps: the row operators together with the head and the verify step."""
import numpy as np
import pytest
import torch

import causal_draft_correction_amd as dca
import domino_synth as ds
from causal_draft_correction_amd import adapt

pytestmark = pytest.mark.gpu

H = 2.0 ** -24
SUM = 140 * H  # a log-sum-exp over float32 logits (derived in test_gpu_rows.py)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dca.load_library()


def small(B, markov=False, K=6, V=3001):
    sh = ds.HeadShape(d=256, h=64, r=32, V=V, K=K, wdtype="bf16")
    w = dca.head_weights_to_device(ds.make_weights(sh, (31, 0), gru_sensitive=True))
    inp = ds.make_inputs(sh, B, (31, 1), sigma=0.5, peak="none")
    args = [dca.device_tensor(x) for x in (inp.H, inp.L_base, inp.last_tok)]
    heads = [dca.DominoHead(w, K=k, max_batch=n, markov=markov) for k, n in ((K, B), (1, 8))]
    return w, heads, args


@pytest.mark.parametrize("markov", [False, True])
def test_one_beam_is_the_greedy_draft(markov):
    """One beam takes each position's largest log-probability: the greedy token (at most 8 rows, where a head gives
    the same bits at any K)."""
    _, (head, one), args = small(3, markov)
    want = head.draft(*args)["tokens"]
    got = adapt.beam_draft(one, *args, beams=1)
    assert torch.equal(got["tokens"][:, 0], want)


@pytest.mark.parametrize("markov", [False, True])
def test_beam_scores_are_sums_of_log_probabilities(markov):
    """Each beam's score against the head's own logits, forced on that beam's tokens; scores fall from beam to beam
    and the best is no worse than the greedy draft's."""
    B, W = 2, 4
    _, (head, one), (Hd, L, last) = small(B, markov)
    K = L.shape[1]
    got = adapt.beam_draft(one, Hd, L, last, beams=W)
    bound = K * (SUM + 40 * H)  # K sums, each rounded to float32 below 2^6
    for j in range(W):
        out = head.draft(Hd, L, last, teacher=got["tokens"][:, j].contiguous(), want_logits=True)
        logp = torch.log_softmax(out["L_final"].double(), -1).gather(2, got["tokens"][:, j].long()[..., None])
        assert (logp.sum((1, 2)) - got["scores"][:, j].double()).abs().max() <= bound
    s = got["scores"].cpu().numpy()
    assert (np.diff(s, axis=1) <= 0).all()
    greedy = adapt.beam_draft(one, Hd, L, last, beams=1)["scores"]
    assert len({tuple(t) for t in got["tokens"][0].tolist()}) == W
    assert (got["scores"][:, 0] - greedy[:, 0]).min() >= -bound


def test_ended_beams_keep_their_score_and_repeat_the_end_token():
    _, (head, one), (Hd, L, last) = small(2)
    eos = int(head.draft(Hd, L, last)["tokens"][0, 1])  # ends the greedy draft at its second token
    got = adapt.beam_draft(one, Hd, L, last, beams=4, eos=eos)
    t = got["tokens"].cpu().numpy()
    ended = np.cumsum(t == eos, 2) > 0
    assert (t[ended] == eos).all() and ended[0].any()


def test_distillation_lowers_the_loss():
    w, _, (Hd, L, last) = small(4)
    g = torch.Generator(device="cuda").manual_seed(3)
    other = (w["W2"].float() + 0.5 * torch.randn(w["W2"].shape, generator=g, device="cuda")).to(torch.bfloat16)
    target = adapt.synthetic_target(w, other, Hd, L, last)
    W2 = torch.nn.Parameter(w["W2"].float().clone())
    optimizer, before, losses = torch.optim.AdamW([W2], lr=0.05), w["W2"].clone(), []
    for _ in range(10):
        losses.append(float(adapt.distill_step(w, W2, Hd, L, last, target, k=32)["loss"]))
        optimizer.step()
    assert torch.equal(w["W2"], before)  # the head's own weights are left alone
    assert np.isfinite(losses).all() and losses[-1] < 0.8 * losses[0], losses


def test_the_example_runs(capsys):
    got = adapt.main(steps=3)
    said = capsys.readouterr().out
    assert "mean accept length" in said and "best of 4 beams" in said
    assert np.isfinite(got["losses"]).all()


def test_beam_draft_refuses_heads_that_do_not_fit():
    _, (head, one), args = small(3)
    with pytest.raises(ValueError, match="K = 1"):
        adapt.beam_draft(head, *args, beams=1)
    with pytest.raises(ValueError, match="max_batch"):
        adapt.beam_draft(one, *args, beams=3)
