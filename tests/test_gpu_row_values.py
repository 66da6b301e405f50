"""Values of the operators over vocabulary rows where rounding, masks or close scores decide them: what one operator
leaves is given to the next, and results are compared with 64-bit forms of their own (H: half a float32 step)."""
import numpy as np
import pytest
import torch

import causal_draft_correction_amd as dca
import rows_plain as plain

pytestmark = pytest.mark.gpu

H = 2.0 ** -24
DTYPES = [torch.float32, torch.bfloat16]
# rows by one block, by one block with the gradient only, and split
LENGTHS = (300, 9001, 70001)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dca.load_library()


def host(t):
    return t.float().cpu().numpy()


def logits(B, R, V, dtype, seed, scale=3.0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn((B, R, V), generator=g).mul_(scale).to(dtype).cuda()


def three_ways(z, ids, values, lse, g, **kw):
    """Loss and gradient by one call, and by a forward and a backward call; the forward call's statistics."""
    both = dca.distill(z, ids, values, lse, grad_loss=g, **kw)
    first = dca.distill(z, ids, values, lse, **kw)
    second = dca.distill_backward(z, ids, first["stats"], g, **kw)
    torch.cuda.synchronize()
    return (both["loss"], both["grad"]), (first["loss"], second), first["stats"]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", LENGTHS)
def test_teacher_rows_whose_mask_leaves_nothing_are_left_out(V, dtype):
    k = 20
    z = logits(1, 4, V, dtype, V)
    target = logits(1, 4, V, torch.float32, V + 1)
    target[0, 1] = -np.inf
    top = dca.top_logits(target, k)
    assert float(top["lse"][0, 1]) == -np.inf and bool((top["ids"][0, 1] >= 0).all())
    g = torch.ones((1, 4), device="cuda")
    for lse in (top["lse"], None):
        one, two, stats = three_ways(z, top["ids"], top["values"], lse, g)
        for loss, grad in (one, two):
            assert float(loss[0, 1]) == 0.0 and not bool(grad[0, 1].float().abs().max() > 0)
            assert bool(torch.isfinite(loss).all()) and bool(torch.isfinite(grad.float()).all())
            assert bool((loss[0, [0, 2, 3]] > 0).all())
        assert not bool(stats[0, 1].abs().max() > 0)
        z2 = z.clone()
        z2[0, 1] = np.nan  # whatever the student's row holds
        again = three_ways(z2, top["ids"], top["values"], lse, g)
        assert torch.equal(again[0][0], one[0]) and torch.equal(again[1][1], two[1])
    # a NaN among the values is no mask
    values = top["values"].clone()
    values[0, 1, 3] = np.nan
    one, two, _ = three_ways(z, top["ids"], values, top["lse"], g)
    assert np.isnan(float(one[0][0, 1])) and np.isnan(float(two[0][0, 1]))


SUM = 140 * H  # a chunk's sum of exponentials, whatever the order of its additions (derived in test_gpu_rows.py)


def certain_rows(B, R, V, dtype, seed, peak=22.0):
    """Rows nearly certain of six ids, and those ids."""
    g = torch.Generator().manual_seed(seed)
    z = torch.randn((B, R, V), generator=g)
    at = torch.stack([torch.randperm(V, generator=g)[:6] for _ in range(B * R)]).view(B, R, 6)
    z.scatter_(2, at, peak - 0.7 * torch.arange(6).float() + torch.randn((B, R, 6), generator=g))
    return z.to(dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("V,k,tau", [(300, 20, 1.0), (9001, 9, 0.7), (70001, 64, 1.442), (40000, 6, 1.0)])
def test_small_losses_of_a_student_that_is_nearly_certain(V, k, tau, tail, dtype):
    """Only the other ids' sum is taken in float32: log q of a named id is off by Qr SUM at most, the loss by the
    masses times that (and rest times the sum's own error), and its rounding; so are the gradients of named ids."""
    check_small_losses(V, k, float(np.float32(tau)), tail, dtype)


@pytest.mark.parametrize("tau", [0.7, 1.442, 1 / 3])
@pytest.mark.parametrize("V", LENGTHS)
def test_temperatures_that_float32_does_not_hold(V, tau):
    """The same bounds: a temperature off by H of itself would move a loss by |log p| H of its masses."""
    check_small_losses(V, 9, tau, True, torch.float32)
    z = logits(1, 3, V, torch.float32, V, 9.0)
    got = host(dca.top_logits(z, 3, temperature=tau)["lse"]).astype(np.float64)
    want = torch.logsumexp(z.double() / tau, -1).cpu().numpy()
    assert (np.abs(got - want) <= 41 * H + np.abs(want) * H).all()


def check_small_losses(V, k, tau, tail, dtype):
    z = certain_rows(2, 4, V, dtype, V + k)
    t = z.float() + 0.05 * torch.randn(z.shape, generator=torch.Generator().manual_seed(k))
    values, ids = t.topk(k)
    lse = torch.logsumexp(t.double() / tau, -1).float() if tail else None
    g = (0.5 + torch.rand((2, 4), generator=torch.Generator().manual_seed(V))).cuda()
    dev = z.cuda()
    one, two, _ = three_ways(dev, ids.int().cuda(), values.cuda(), None if lse is None else lse.cuda(), g,
                             temperature=tau)
    loss, grad, _ = plain.distill(z.float().numpy(), ids.numpy(), values.numpy(),
                                  None if lse is None else lse.numpy(), tau)
    y = z.double() / tau
    q = torch.softmax(y, -1)
    other = (1.0 - q.gather(2, ids).sum(-1)).clamp(min=0).numpy() + 1e-15
    rest = np.zeros((2, 4)) if lse is None else np.maximum(0, 1 - np.exp(
        values.numpy().astype(np.float64) / tau - lse.numpy()[..., None].astype(np.float64)).sum(-1))
    most = tau * tau * SUM * (2 * other + 2 * rest) + np.abs(loss) * H + 1e-13
    named = np.take_along_axis(grad, ids.numpy(), 2) * g.cpu().numpy()[..., None].astype(np.float64)
    qn = q.gather(2, ids).numpy()
    for got, gr in (one, two):
        assert (np.abs(host(got).astype(np.float64) - loss) <= most).all(), np.abs(host(got) - loss).max()
        if dtype == torch.float32:
            off = np.abs(np.take_along_axis(host(gr).astype(np.float64), ids.numpy(), 2) - named)
            # h, grad_loss * tau and their product are rounded to float32 (tau is: H of the product)
            assert (off <= 1.5 * tau * qn * other[..., None] * SUM + 4 * H * np.abs(named) + 1e-13).all(), off.max()


def noise_of(lse):
    """What a float32 log-sum-exp leaves open of a mass (include/domino_head.h)."""
    return (np.abs(lse.astype(np.float64)) + 32) * H


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V,k,left,tau,fill", [
    (7, 7, 7, 1.0, None), (50, 50, 50, 0.5, None), (128, 128, 128, 2.0, None),
    *[(V, k, left, 1.0, fill) for V, k, left in ((2000, 64, 40), (20000, 128, 100), (70001, 64, 5))
      for fill in ("-inf", "lowest")]])
def test_a_student_that_is_its_teacher_where_the_entries_hold_all_there_is(V, k, left, tau, fill, dtype):
    """Masses brought to a sum of 1 and a sum of q that is all named: equal in 64 bits, whatever way the teacher's
    log-sum-exp was rounded."""
    z = logits(8, 25, V, dtype, V + k)
    if fill:
        at = torch.rand((8, 25, V), generator=torch.Generator().manual_seed(k)).argsort(-1)[..., :left].cuda()
        x = torch.full_like(z, -np.inf if fill == "-inf" else torch.finfo(dtype).min)
        z = x.scatter(2, at, z.gather(2, at))
    top = dca.top_logits(z, k, temperature=tau)
    g = torch.ones((8, 25), device="cuda")
    one, two, _ = three_ways(z, top["ids"], top["values"], top["lse"], g, temperature=tau)
    for loss, grad in (one, two):
        assert float(loss.abs().max()) <= 1e-12
        assert float(grad.float().abs().max()) <= 1e-12


@pytest.mark.parametrize("V,k", [(2000, 64), (9001, 128), (70001, 64)])
@pytest.mark.parametrize("tau", [1.0, 0.1, 0.05, 0.01, 0.001])
def test_top_logits_into_distill_at_low_temperatures(V, k, tau):
    """Against the loss with the teacher's log-sum-exp in 64 bits: a mass is off by the noise of L (the other ids' by
    that too), and x log(x / Qr) over such a step, or up to twice that where a row counts as without L, by the step
    times |log Qr| + |log noise| + 1.  For a student that is its teacher x is at most Qr + noise: below twice the noise
    times 1 + |log noise| while Qr exceeds noise^2, and no such term below."""
    tau = float(np.float32(tau))
    target = logits(1, 6, V, torch.float32, V, 4.0)
    g = torch.ones((1, 6), device="cuda")
    top = dca.top_logits(target, k, temperature=tau)
    ids = top["ids"].long()
    noise = noise_of(host(top["lse"]))
    t = target.double() / tau
    logp = torch.log_softmax(t, -1)

    def other_mass(y):  # log of the other ids' sum
        return y.scatter(2, ids, -np.inf).logsumexp(-1)

    log_rest = other_mass(logp)
    for name, z in (("itself", target), ("another", logits(1, 6, V, torch.float32, V + 1, 1.0) + target)):
        logq = torch.log_softmax(z.double() / tau, -1)
        log_qr = other_mass(logq)
        p, lq = logp.gather(2, ids).exp(), logq.gather(2, ids)
        terms = torch.where(p > 0, p * (logp.gather(2, ids) - lq), 0.0)
        rest = log_rest.exp()
        want = (terms.sum(-1) + torch.where(rest > 0, rest * (log_rest - log_qr), 0.0)).cpu().numpy()
        if name == "itself":
            most = 2 * noise * (1 + np.abs(np.log(noise))) + 2 * SUM * rest.cpu().numpy()
        else:
            size = (terms.abs().sum(-1) + log_qr.abs()).cpu().numpy()
            most = 2 * noise * (size + 3 + np.abs(np.log(noise))) + 2 * SUM + np.abs(want) * H
        one, two, _ = three_ways(z, top["ids"], top["values"], top["lse"], g, temperature=tau)
        for loss, grad in (one, two):
            off = np.abs(host(loss).astype(np.float64) / tau ** 2 - want)
            assert (off <= most).all(), (name, off, most)
            if name == "itself":
                assert (np.abs(host(grad) / tau).max(-1) <= 4 * noise + 2 * SUM).all(), name


def test_sums_of_beams_keep_what_other_threads_add():
    """One logit of 0 and one of -25 log 2, in another thread of the same wave, another wave or another chunk: the
    sum is 1 + 2^-25, of which float32 leaves nothing.  The exponential is good to 2 H and its argument to 25 log2(e) H
    (fused, rounded once: less than 32 H); log(1 + x) = x within x^2."""
    V, low, small = 40000, -25 * np.log(2.0), 2.0 ** -25
    for far in (8, 300, 20000, 39999):
        z = torch.full((1, 2, V), -np.inf)
        z[0, :, 0] = 0.0
        z[0, 0, far] = low
        x = float(np.exp(np.float64(np.float32(low))))  # what the float32 logit stands for
        lse = float(dca.top_logits(z.cuda(), 2)["lse"][0, 0])
        assert abs(lse - np.log1p(x)) <= 64 * H * small, far
        # -2^-25 against -1e-8: the second beam's only token is the better one
        got = dca.beam_step(z.cuda(), torch.tensor([[0.0, -1e-8]]).cuda(), n_out=2)
        assert got["parent"][0].tolist() == [1, 0] and got["token"][0].tolist() == [0, 0], far
        assert float(got["scores"][0, 0]) == np.float32(-1e-8)
        assert abs(float(got["scores"][0, 1]) + np.log1p(x)) <= 64 * H * small, far


@pytest.mark.parametrize("V", [300, 40000])
def test_gradients_beside_the_logits_in_one_buffer(V):
    z = logits(2, 3, V, torch.float32, V)
    top = dca.top_logits(z + 1.0, 8)
    teach = dict(ids=top["ids"], values=top["values"], teacher_lse=top["lse"], grad_loss=torch.ones((2, 3), device="cuda"))
    want = dca.distill(z, **teach)["grad"]
    room = torch.cat([z, torch.zeros_like(z)], -1)  # the right half of every row
    got = dca.distill(room[..., :V], out={"grad": room[..., V:]}, **teach)["grad"]
    assert torch.equal(got, want) and torch.equal(room[..., :V], z)
    room = torch.stack([z, torch.zeros_like(z)])  # one behind the other
    assert torch.equal(dca.distill(room[0], out={"grad": room[1]}, **teach)["grad"], want)
    # one row of each batch entry, and one entry: the stride of a dimension of length 1 says nothing
    one = {n: x[:, :1].contiguous() for n, x in teach.items()}
    own = z[:, :1].clone()
    place = torch.as_strided(own, (2, 1, V), (V, 3, 1))
    assert torch.equal(dca.distill(own, out={"grad": place}, **one)["grad"], want[:, :1])
    for shift in (1, V - 1):
        with pytest.raises(dca.DominoError, match="overlaps"):
            flat = torch.zeros(6 * V + V, device="cuda")
            dca.distill(flat[:6 * V].view(2, 3, V), out={"grad": flat[shift:shift + 6 * V].view(2, 3, V)}, **teach)


def test_logits_that_require_a_gradient():
    """A loss without a graph is not handed out in its place; the gradient that the operator computes can go on."""
    z = logits(2, 3, 500, torch.float32, 1)
    top = dca.top_logits(z + 1.0, 8)
    leaf = z.clone().requires_grad_()
    teach = dict(ids=top["ids"], values=top["values"], teacher_lse=top["lse"])
    with pytest.raises(ValueError, match="detach"):
        dca.distill(leaf, **teach)
    with torch.no_grad():
        first = dca.distill(leaf, **teach)
    g = torch.ones((2, 3), device="cuda")
    two = dca.distill_backward(leaf, top["ids"], first["stats"], g)
    leaf.backward(dca.distill(leaf, grad_loss=g, **teach)["grad"])
    assert torch.equal(leaf.grad, two) and torch.equal(two, dca.distill(z, grad_loss=g, **teach)["grad"])


@pytest.mark.parametrize("V", LENGTHS)
def test_loss_without_statistics(V):
    z = logits(2, 3, V, torch.bfloat16, V)
    top = dca.top_logits(logits(2, 3, V, torch.float32, V + 1), 12)
    want = dca.distill(z, top["ids"], top["values"], top["lse"])
    got = dca.distill(z, top["ids"], top["values"], top["lse"], want_stats=False)
    assert set(got) == {"loss"} and torch.equal(got["loss"], want["loss"])
    with pytest.raises(ValueError, match="out"):
        dca.distill(z, top["ids"], top["values"], out={"stats": want["stats"]}, want_stats=False)


def candidate_scores(z, scores, eos, finished):
    """[W, V] of one batch entry, in 64 bits, from the definition."""
    out = np.full(z.shape, -np.inf)
    for w, row in enumerate(z.astype(np.float64)):
        s = float(scores[w])
        if s == -np.inf:
            continue
        if finished is not None and finished[w]:
            out[w, eos] = s
        elif not s < np.inf or np.isnan(row).any() or (row == np.inf).any():
            out[w] = np.nan
        elif (row > -np.inf).any():
            out[w] = s + plain.log_softmax(row)
    return out


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,W,V,M,eos", [
    (3, 1, 2, 1, -1), (2, 4, 700, 1, -1), (2, 4, 5003, 1, 5), (1, 32, 3000, 1, 2999), (1, 4, 151936, 1, -1),
    (4, 6, 40001, 1, 0), (2, 4, 151936, 8, 7), (1, 32, 4099, 128, 3), (9, 5, 20011, 17, -1), (3, 3, 50, 100, 49)])
def test_every_beam_has_the_score_of_its_parent_and_token(B, W, V, M, eos, dtype):
    """Each place by its own candidate's score, the last one too: it is the reported one within a sum's bound and its
    rounding, and the one that belongs in that place within twice the bound."""
    g = torch.Generator().manual_seed(V + M)
    z = logits(B, W, V, dtype, V)
    scores = -torch.cumsum(0.1 + torch.rand((B, W), generator=g), 1)
    finished = torch.rand((B, W), generator=g) < 0.3 if eos >= 0 else None
    scores[:, W // 2 + 1:][torch.rand(scores[:, W // 2 + 1:].shape, generator=g) < 0.2] = -np.inf
    state = torch.randn((B, W, 12), generator=g)
    history = torch.randint(0, V, (B, W, 3), generator=g, dtype=torch.int32)
    got = dca.beam_step(z, scores.cuda(), n_out=M, eos=eos, finished=None if eos < 0 else finished.cuda(),
                        state=state.cuda(), history=history.cuda(), step=1)
    torch.cuda.synchronize()
    p, t, s = (got[n].cpu().numpy() for n in ("parent", "token", "scores"))
    for b in range(B):
        each = candidate_scores(host(z[b]), scores[b].numpy(), eos, None if eos < 0 else finished[b].numpy())
        own = each[p[b], t[b]]
        want = np.sort(each.reshape(-1))[::-1][:M]
        assert len({*zip(p[b], t[b])}) == M
        fine = np.isfinite(want)
        assert np.array_equal(np.isneginf(own), np.isneginf(want)) and np.array_equal(np.isneginf(s[b]), ~fine)
        assert (np.abs(own[fine] - want[fine]) <= 2 * SUM).all()
        assert (np.abs(s[b][fine] - own[fine]) <= SUM + np.abs(own[fine]) * H).all()
        assert np.array_equal(got["state"][b].cpu().numpy(), state[b].numpy()[p[b]])
        moved = history[b].numpy()[p[b]]
        moved[:, 1] = t[b]
        assert np.array_equal(got["history"][b].cpu().numpy(), moved)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", LENGTHS)
@pytest.mark.parametrize("tau", [2.0, 1.0, 0.5, 1e-4])
def test_teacher_rows_at_the_lowest_value(V, tau, dtype):
    """Their log-sum-exp is -3e38, or -inf in float32: nothing of it can be the other ids', so they are rows without it.
    So is a row whose temperature leaves of it less than a mass of 2^-6 can be told by."""
    k, tau = 20, float(np.float32(tau))
    z = logits(1, 4, V, dtype, V)
    target = logits(1, 4, V, dtype, V + 1)
    target[0, 1] = torch.finfo(dtype).min
    target[0, 2] = 40.0
    target[0, 2, V // 2] = 41.0
    top = dca.top_logits(target, k, temperature=tau)
    assert float(top["lse"][0, 1]) <= -3e38 / max(1.0, tau)
    g = torch.ones((1, 4), device="cuda")
    blind = [1] + ([2] if tau < 1e-3 else [])
    told = three_ways(z, top["ids"], top["values"], top["lse"], g, temperature=tau)
    alone = three_ways(z, top["ids"], top["values"], None, g, temperature=tau)
    for (loss, grad), (want, want_grad) in zip(told[:2], alone[:2]):
        assert bool(torch.isfinite(loss).all()) and bool(torch.isfinite(grad.float()).all())
        for r in blind:
            assert torch.equal(loss[0, r], want[0, r]) and torch.equal(grad[0, r], want_grad[0, r])
        if tau > 1e-3:
            assert not torch.equal(loss[0, 2], want[0, 2])  # (most of this row's mass is the other ids')
    # a row of equal values over k entries: log(1 / k) - mean log q
    logq = torch.log_softmax(z.double() / tau, -1)[0, 1].gather(0, top["ids"][0, 1].long())
    want = float(tau ** 2 * (-np.log(k) - logq.mean()))
    assert abs(float(told[0][0][0, 1]) - want) <= 2 * tau ** 2 * SUM + 2 * abs(want) * H


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,R,V,tau", [(1, 1, 300, 1.0), (40, 3, 2049, 0.7), (2, 2, 32000, 1.442), (300, 2, 16385, 1.0),
                                       (2, 3, 151936, 1.442), (1, 1, 524288, 2.0)])
def test_log_sum_exps_by_the_depth_of_their_sums(B, R, V, tau, dtype):
    """Half steps of a sum: 2 of an exponential; the rounding of its argument, and that of log2(e) / tau, |d| of a term
    exp(-d) each, which over 2^19 terms is 9.8 of the sum at most; 19 additions of a thread (4 elements, 16 vectors),
    and none after, in 64 bits.  41 H, and the result's rounding."""
    tau = float(np.float32(tau))
    for scale in (0.01, 1.0, 3.0, 9.0):
        z = logits(B, R, V, dtype, V + int(scale), scale)
        got = host(dca.top_logits(z, 3, temperature=tau)["lse"]).astype(np.float64)
        want = torch.logsumexp(z.double() / tau, -1).cpu().numpy()
        assert (np.abs(got - want) <= 41 * H + np.abs(want) * H).all(), (scale, np.abs(got - want).max() / H)
