"""GPU results of the operators over vocabulary rows against their plain 64-bit forms (rows_plain.py).

Bounds, in halves of a float32 step (H = 2^-24, torch.finfo(float32).eps / 2).  A thread adds at most 128
exponentials, so at most 128 H whatever the order of its sum, and a wave joins 64 sums in 6 steps (6 H); chunks are
joined in 64 bits.  An exponential has one step of its own (2 H) and the rounding of its argument, |d| log2(e) H for
d = z - m, which with terms exp(-|d|) weighs less than 1 H in a sum.  The factor log2(e) / tau is rounded for
arguments below 1024: |log2 q| ln 2 H / 2 in a term q, at most log2(V) ln 2 / 2 < 7 H in a sum.  A sum vector by
vector has a depth of 22, not 128, so SUM = 140 H holds all of this for a log-sum-exp, before it is rounded to
float32 (|lse| H).
"""
import numpy as np
import pytest
import torch

import causal_draft_correction_amd as dca
import rows_plain as plain

pytestmark = pytest.mark.gpu

H = 2.0 ** -24
SUM = 140 * H
HALF = {torch.float32: H, torch.bfloat16: 2.0 ** -8}
DTYPES = [torch.float32, torch.bfloat16]


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


def same_nan(a, b):
    return np.array_equal(np.isnan(a), np.isnan(b))


def check_top(z, k, tau, n_rows=None, label=""):
    nr = None if n_rows is None else torch.tensor(n_rows, dtype=torch.int32, device="cuda")
    got = dca.top_logits(z, k, temperature=tau, n_rows=nr)
    again = dca.top_logits(z, k, temperature=tau, n_rows=nr)
    torch.cuda.synchronize()
    ids, values, lse = plain.top(host(z), k, tau, n_rows)
    assert np.array_equal(got["ids"].cpu().numpy(), ids), label
    v, l = host(got["values"]), host(got["lse"])
    assert np.array_equal(v, values, equal_nan=True), label
    assert same_nan(l, lse), label
    inf = np.isinf(lse)
    assert np.array_equal(l[inf], lse[inf]), label
    fine = np.isfinite(lse)
    assert (np.abs(l[fine] - lse[fine]) <= SUM + np.abs(lse[fine]) * H).all(), label
    for name in got:
        assert got[name].cpu().numpy().tobytes() == again[name].cpu().numpy().tobytes(), label


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,R,V,k,pad,shift,tau", [
    (1, 1, 1, 1, 0, 0, 1.0), (1, 3, 7, 7, 0, 1, 1.0), (2, 3, 130, 5, 3, 0, 0.5), (1, 2, 1024, 128, 0, 0, 1.0),
    (2, 1, 1025, 64, 0, 3, 2.0), (1, 1, 2048, 1, 5, 1, 1.0), (3, 2, 5003, 33, 0, 0, 1.0), (1, 1, 16384, 128, 0, 0, 1.0),
    (2, 2, 16385, 100, 7, 1, 0.7), (1, 2, 40001, 128, 0, 0, 1.0), (1, 1, 151936, 64, 0, 0, 1.0),
    (200, 4, 2500, 3, 0, 1, 1.0), (30, 40, 4099, 17, 1, 0, 1.0), (1, 1, 524288, 128, 0, 0, 1.0),
    (1, 2, 32768, 128, 0, 0, 1.0), (1, 1, 32769, 7, 0, 1, 1.0), (70, 4, 20011, 33, 0, 0, 1.0),
    (3, 1, 65536, 100, 0, 0, 2.0), (2, 1, 65537, 5, 3, 0, 1.0),
])
def test_top_logits(B, R, V, k, pad, shift, tau, dtype):
    check_top(rows(B, R, V, dtype, 7 * V + k, pad, shift), k, tau, label="B=%d R=%d V=%d k=%d" % (B, R, V, k))


def special_rows(V, dtype):
    """Rows with masks that leave little or nothing, infinities, NaN, ties and sorted orders, by name."""
    g = torch.Generator().manual_seed(V)
    base = torch.randn(V, generator=g) * 3
    low = torch.finfo(dtype).min
    out = {"all -inf": torch.full((V,), -np.inf), "all lowest": torch.full((V,), low), "all zero": torch.zeros(V)}
    for name, fill in (("five left, -inf", -np.inf), ("five left, lowest", low)):
        x = torch.full((V,), fill)
        at = torch.randperm(V, generator=g)[:5]
        x[at] = base[at]
        out[name] = x
    x = torch.full((V,), -np.inf)
    x[V - 1] = -1.5
    out["last one left"] = x
    x = torch.full((V,), -np.inf)
    x[::2] = base[::2]
    out["half masked"] = x
    x = base.clone()
    x[V // 3], x[2 * V // 3] = np.nan, np.nan
    out["NaN"] = x
    x = base.clone()
    x[V // 2], x[V - 1] = np.inf, np.inf
    out["+inf"] = x
    x = base.clone()
    x[0], x[V // 2] = np.inf, np.nan
    out["NaN and +inf"] = x
    x = torch.zeros(V)
    x[: V // 2] = -0.0
    out["+-0"] = x
    out["ascending"] = torch.arange(V).float()
    out["descending"] = -torch.arange(V).float()
    out["few values"] = torch.randint(0, 3, (V,), generator=g).float()
    # three waves of every four hold large values, the fourth small ones: a wave's share is no guide to the row's
    vec = 4 if dtype == torch.float32 else 8
    quiet = (torch.arange(V) // vec) % 256 < 64
    out["one quiet wave"] = torch.where(quiet, base.abs() * -1.0, 100.0 + base.abs())
    x = torch.full((V,), -np.inf)
    x[V // 3:V // 3 + min(V // 2, 2500)] = base[V // 3:V // 3 + min(V // 2, 2500)]
    out["neighbours left"] = x
    x = torch.full((V,), 2.0)
    x[V // 7::V // 7] = 3.0
    out["ties below a few"] = x
    return {name: row.to(dtype) for name, row in out.items()}


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V,k", [(300, 128), (2100, 100), (16000, 64), (30001, 100), (70000, 128)])
def test_top_logits_of_special_rows(V, k, dtype):
    named = special_rows(V, dtype)
    for name, row in named.items():
        check_top(row.cuda().view(1, 1, V), k, 1.0, label=name)
    check_top(torch.stack(list(named.values())).cuda().view(1, len(named), V), k, 1.5, label="together")


def test_top_logits_lengths_strides_and_two_dimensions():
    wide = rows(4, 6, 3001, torch.float32, 5)
    check_top(wide[:, :5], 9, 1.0, [0, 1, 5, 99], "slice of rows")          # batch stride of 6 rows
    check_top(wide[:, 1:2].expand(4, 3, 3001), 9, 1.0, None, "one row for all")
    check_top(wide.transpose(0, 1), 4, 1.0, None, "batch and rows exchanged")
    check_top(wide[:1], 4, 1.0, [-3], "negative length")
    two = dca.top_logits(wide[0], 9)
    three = dca.top_logits(wide[:1], 9)
    for name in two:
        assert torch.equal(two[name], three[name][0]), name
    none = dca.top_logits(wide[:0], 9)
    assert none["ids"].shape == (0, 6, 9)


def test_rows_past_31_bit_offsets():
    """Batch entries more than 2^31 elements apart."""
    V, far = 5001, 2 ** 31 + 24
    big = torch.zeros(far + 2 * V, dtype=torch.bfloat16, device="cuda")
    z = torch.as_strided(big, (2, 2, V), (far, V, 1))
    z.copy_(rows(2, 2, V, torch.bfloat16, 11))
    check_top(z, 20, 1.0)
    ids, values, lse = plain.top(host(z), 20, 1.0)
    teach = dict(ids=torch.tensor(ids, dtype=torch.int32, device="cuda"),
                 values=torch.tensor(values, dtype=torch.float32, device="cuda"))
    g = torch.ones((2, 2), device="cuda")
    want = dca.distill(z.contiguous(), grad_loss=g, **teach)
    got = dca.distill(z, grad_loss=g, out={"grad": z}, **teach)
    assert torch.equal(got["loss"], want["loss"]) and torch.equal(got["grad"].contiguous(), want["grad"])


# ---- beam_step ----

def check_beam(z, scores, M, eos=-1, finished=None, state=None, history=None, step=0, label=""):
    dev = lambda x: None if x is None else x.cuda()  # noqa: E731
    args = dict(n_out=M, eos=eos, finished=dev(finished), state=dev(state), history=dev(history), step=step)
    got = dca.beam_step(z, scores.cuda(), **args)
    again = dca.beam_step(z, scores.cuda(), **args)
    torch.cuda.synchronize()
    want, parent, token = plain.beam(host(z), scores.numpy(), M, eos, None if finished is None else finished.numpy())
    s = host(got["scores"]).astype(np.float64)
    assert same_nan(s, want), label
    inf = np.isinf(want)
    assert np.array_equal(s[inf], want[inf]), label
    fine = np.isfinite(want)
    assert (np.abs(s[fine] - want[fine]) <= SUM + np.abs(want[fine]) * H).all(), label
    # the same candidates in the same places, but where two scores lie within the bound of each other
    p, t = got["parent"].cpu().numpy(), got["token"].cpu().numpy()
    B = z.shape[0]
    for b in range(B):
        for j in np.flatnonzero((p[b] != parent[b]) | (t[b] != token[b])):
            near = [abs(want[b, j] - want[b, i]) for i in (j - 1, j + 1) if 0 <= i < M]
            assert fine[b, j] and (j == M - 1 or min(near) <= 2 * SUM), (label, b, j)
        assert len({(x, y) for x, y in zip(p[b], t[b])}) == M, label
    if eos >= 0:
        ended = t == eos
        if finished is not None:
            ended |= np.take_along_axis(finished.numpy(), p.astype(np.int64), 1)
        assert np.array_equal(got["finished"].cpu().numpy(), ended), label
    if state is not None:
        for b in range(B):
            assert torch.equal(got["state"][b].cpu(), state[b][torch.tensor(p[b]).long()]), label
    if history is not None:
        for b in range(B):
            h = history[b][torch.tensor(p[b]).long()].clone()
            h[:, step] = torch.tensor(t[b])
            assert torch.equal(got["history"][b].cpu(), h), label
    for name in got:
        assert torch.equal(got[name].view(torch.uint8), again[name].view(torch.uint8)), label
    return got


def some_scores(B, W, seed):
    g = torch.Generator().manual_seed(seed)
    return -torch.cumsum(0.1 + torch.rand((B, W), generator=g), 1)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,W,V,M,h,pad,shift", [
    (1, 1, 1, 1, 1, 0, 0), (2, 3, 2, 6, 5, 0, 1), (1, 4, 1024, 4, 64, 0, 0), (3, 5, 1001, 9, 12, 3, 1),
    (2, 8, 5003, 16, 1024, 0, 0), (1, 32, 4099, 128, 33, 1, 0), (1, 4, 151936, 8, 256, 0, 0),
    (40, 7, 2051, 13, 20, 0, 0), (2, 2, 90001, 2, 40000, 0, 1),
])
def test_beam_step(B, W, V, M, h, pad, shift, dtype):
    g = torch.Generator().manual_seed(V + W)
    z = rows(B, W, V, dtype, 13 * V + W, pad, shift)
    scores, state = some_scores(B, W, V), torch.randn((B, W, h), generator=g)
    history = torch.randint(0, V, (B, W, 5), generator=g, dtype=torch.int32)
    check_beam(z, scores, M, state=state, history=history, step=3)
    finished = torch.rand((B, W), generator=g) < 0.4
    check_beam(z, scores, M, eos=V // 2, finished=finished, state=state.to(torch.bfloat16)
               if h % 2 == 0 else state, history=history, step=0)
    scores[:, 1:] = -np.inf  # the first step: one live beam
    check_beam(z, scores, M, eos=0)


@pytest.mark.parametrize("dtype", DTYPES)
def test_beam_step_of_special_rows(dtype):
    for V, M in ((40, 24), (5000, 20)):
        named = special_rows(V, dtype)
        for name, row in named.items():
            z = torch.stack([row, special_rows(V, dtype)["half masked"], row]).cuda().view(1, 3, V)
            for scores in ([-1.0, -2.0, -1.0], [-np.inf, -1.0, -2.0], [-np.inf] * 3, [np.nan, -1.0, -2.0],
                           [-1.0, np.inf, -2.0]):
                check_beam(z, torch.tensor([scores]), M, label="%s %s" % (name, scores))
            check_beam(z, torch.tensor([[-1.0, -3.0, -2.0]]), M, eos=3, label=name + " ended",
                       finished=torch.tensor([[True, False, False]]))
            check_beam(z, torch.tensor([[-1.0, -3.0, -np.inf]]), M, eos=V - 1, label=name + " all ended",
                       finished=torch.tensor([[True, True, True]]))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,W,V,M", [(2, 4, 700, 8), (1, 32, 3000, 128), (2, 8, 40000, 16), (1, 3, 50, 100)])
def test_beam_step_with_little_left_or_much_equal(B, W, V, M, dtype):
    base = rows(B, W, V, dtype, V + M)
    scores = some_scores(B, W, M)
    first = torch.full_like(scores, -np.inf)
    first[:, W // 2] = -0.5
    for left in (1, 3, min(200, V - 7)):
        z = torch.full_like(base, -np.inf)
        z[..., 7:7 + left] = base[..., 7:7 + left]
        check_beam(z, scores, M, label="%d tokens left" % left)
        check_beam(z, first, M, label="%d tokens left of one beam" % left)
    zero = torch.zeros_like(base)
    zero[..., 3] = -np.inf
    lowest, nan = torch.full_like(scores, torch.finfo(torch.float32).min), scores.clone()
    nan[:, W - 1] = np.nan
    ended = torch.ones((B, W), dtype=torch.bool)
    some = torch.arange(W).expand(B, W) % 2 == 1
    # equal scores have an order: these are the same candidates in the same places
    for label, z, sc, end in (("equal logits", zero, scores, None), ("all equal", zero, torch.ones_like(scores), None),
                              ("lowest scores", base, lowest, None), ("all ended", base, scores, ended),
                              ("all ended, equal scores", base, torch.ones_like(scores), ended),
                              ("some ended, equal logits", zero, torch.ones_like(scores), some),
                              ("a NaN score among ended ones", base, nan, ended), ("a NaN score", zero, nan, None)):
        eos = -1 if end is None else 5
        got = check_beam(z, sc, M, eos=eos, finished=end, label=label)
        _, parent, token = plain.beam(host(z), sc.numpy(), M, eos, None if end is None else end.numpy())
        assert np.array_equal(got["parent"].cpu().numpy(), parent), label
        assert np.array_equal(got["token"].cpu().numpy(), token), label


def test_beam_step_does_not_read_dead_and_ended_rows():
    z = rows(1, 3, 3000, torch.float32, 3)
    scores = torch.tensor([[-1.0, -np.inf, -0.5]])
    finished = torch.tensor([[False, False, True]])
    a = check_beam(z, scores, 6, eos=1, finished=finished)
    z[0, 1:] = np.nan
    b = check_beam(z, scores, 6, eos=1, finished=finished)
    for name in a:
        assert torch.equal(a[name], b[name]), name


# ---- distill ----

def teacher(z, k, tau, tail, seed):
    """A teacher near the student z: its top k logits and, with tail, its log-sum-exp."""
    g = torch.Generator().manual_seed(seed)
    t = torch.tensor(host(z)) + torch.randn(z.shape, generator=g)
    values, ids = t.topk(k)
    lse = torch.logsumexp(t.double() / tau, -1).float() if tail else None
    return ids.int().contiguous(), values.contiguous(), lse


def check_distill(z, ids, values, lse, tau, n_rows=None, label=""):
    dtype, k = z.dtype, ids.shape[-1]
    B, R, V = z.shape
    dev = lambda x: None if x is None else x.cuda()  # noqa: E731
    g = torch.rand((B, R), generator=torch.Generator().manual_seed(k)) + 0.5
    g.view(-1)[::5] *= -1
    nr = None if n_rows is None else torch.tensor(n_rows, dtype=torch.int32, device="cuda")
    teach = dict(ids=dev(ids), values=dev(values), teacher_lse=dev(lse), temperature=tau, n_rows=nr)
    both = dca.distill(z, grad_loss=dev(g), **teach)
    first = dca.distill(z, **teach)
    second = dca.distill_backward(z, dev(ids), first["stats"], dev(g), temperature=tau, n_rows=nr)
    torch.cuda.synchronize()
    with np.errstate(invalid="ignore"):
        loss, grad, size = plain.distill(host(z), ids.numpy(), values.numpy(), None if lse is None else lse.numpy(),
                                         tau, n_rows)
        inf, fine = np.isinf(loss), np.isfinite(loss)
        # p weighs log q (SUM), rest weighs log Qr (two sums); masses sum to 1 (or to the sum of the p)
        t = values.numpy().astype(np.float64) / tau
        mass = np.ones((B, R)) if lse is None else np.maximum(1, np.exp(t - lse.numpy()[..., None]).sum(-1))
        most = 2 * tau * tau * SUM * mass + np.abs(loss) * H
        for name, res in (("both", both["loss"]), ("first", first["loss"])):
            got = host(res).astype(np.float64)
            assert same_nan(got, loss), (label, name)
            assert np.array_equal(got[inf], loss[inf]), (label, name)
            assert (np.abs(got[fine] - loss[fine]) <= most[fine]).all(), (label, name)
        # an element: its sums (q: one, q / Qr and Qr: one each), its exponential (2 H, and the rounding of an
        # argument of at most 88 / log2(e) in size, both products), four products and A's rounding
        rel = 2 * SUM + 2 * H + 2 * 128 * H + 6 * H
        # (exponentials below 2^-126 are 0)
        bound = np.abs(g.numpy())[..., None] * (size * rel + 8 * 2.0 ** -126)
        want = grad * g.numpy()[..., None].astype(np.float64)
        for name, res in (("both", both["grad"]), ("two", second)):
            e = host(res).astype(np.float64)
            assert same_nan(e, want), (label, name)
            ok = np.isfinite(want)
            off = np.abs(e - want) - bound - np.abs(want) * HALF[dtype] * (1 + rel)
            assert (off[ok] <= 0).all(), (label, name, off[ok].max())
    own = z.clone()  # in the logits' place
    place = dca.distill(own, grad_loss=dev(g), out={"grad": own}, **teach)
    assert place["grad"].data_ptr() == own.data_ptr()
    assert torch.equal(own.view(torch.uint8), both["grad"].view(torch.uint8)), label


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("B,R,V,k,pad,shift,tau", [
    (1, 1, 1, 1, 0, 0, 1.0), (2, 2, 7, 7, 0, 1, 1.0), (1, 3, 130, 5, 3, 0, 0.5), (2, 2, 1024, 128, 0, 0, 1.0),
    (2, 1, 1025, 64, 0, 3, 2.0), (3, 2, 5003, 33, 1, 0, 1.0), (1, 1, 16384, 1, 0, 0, 1.0),
    (1, 2, 40001, 100, 7, 1, 3.0),
    (1, 1, 151936, 64, 0, 0, 1.0), (33, 40, 2049, 8, 0, 0, 1.0), (13, 16, 20011, 9, 0, 1, 1.0),
    (1, 2, 32768, 17, 0, 0, 1.0), (1, 1, 32769, 3, 0, 1, 1.0), (9, 31, 16411, 33, 0, 0, 2.0),
    (1, 2, 65551, 128, 3, 0, 1.0),
])
def test_distill(B, R, V, k, pad, shift, tau, tail, dtype):
    z = rows(B, R, V, dtype, 3 * V + k, pad, shift)
    check_distill(z, *teacher(z, k, tau, tail, V), tau, label="B=%d R=%d V=%d k=%d" % (B, R, V, k))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tail", [False, True])
def test_distill_of_special_rows(tail, dtype):
    for V, k in ((300, 20), (9001, 128), (70001, 40)):
        named = special_rows(V, dtype)
        z = torch.stack(list(named.values())).cuda().view(1, len(named), V)
        calm = rows(1, len(named), V, dtype, 1)
        check_distill(z, *teacher(calm, k, 1.0, tail, 5), 1.0, label="special student, V=%d" % V)
        own = plain.top(host(z), k, 1.0)  # the student's own rows as the teacher's
        fine = np.isfinite(own[2])
        ids, values = torch.tensor(own[0], dtype=torch.int32), torch.tensor(own[1], dtype=torch.float32)
        lse = torch.tensor(own[2], dtype=torch.float32)[:, fine[0]].contiguous() if tail else None
        sel = torch.tensor(np.flatnonzero(fine[0]))
        check_distill(z[:, sel.cuda()], ids[:, sel].contiguous(), values[:, sel].contiguous(), lse, 1.0,
                      label="itself, V=%d" % V)


@pytest.mark.parametrize("tail", [False, True])
def test_distill_entries_padded_repeated_and_left_out(tail):
    z = rows(3, 4, 2500, torch.float32, 21)
    ids, values, lse = teacher(z, 9, 1.0, tail, 4)
    ids[0, 0, 3:] = -1                 # fewer entries
    ids[0, 1] = -1                     # none
    ids[0, 2, 0], ids[0, 2, 1] = 2500, 2 ** 31 - 1   # past the vocabulary
    ids[1, 0, 4] = ids[1, 0, 2]        # named twice
    ids[1, 1] = ids[1, 1, 0]           # one id nine times
    values[1, 2, 5:] = -np.inf         # entries without mass
    if not tail:
        values[1, 3] = -np.inf         # no mass at all
    check_distill(z, ids, values, lse, 1.0)
    check_distill(z, ids, values, lse, 1.0, [0, 3, 99])
    z[0, 1], z[1, 3] = np.nan, np.nan  # rows left out are not read
    got = dca.distill(z, ids.cuda(), values.cuda(), None if lse is None else lse.cuda(),
                      n_rows=torch.tensor([2, 3, 4], dtype=torch.int32, device="cuda"),
                      grad_loss=torch.ones((3, 4), device="cuda"))
    assert not torch.isnan(got["loss"]).any() and not torch.isnan(got["grad"]).any()


def test_distill_masses_that_exceed_one_and_a_certain_student():
    z = rows(1, 3, 4000, torch.float32, 8, scale=1.0)
    ids, values, lse = teacher(z, 5, 1.0, True, 4)
    lse[0, 0] -= 3.0                       # the entries' masses sum to more than 1
    z[0, 1] *= 0.01
    z[0, 1, ids[0, 1].long().cuda()] = 200.0    # all else has less mass than float32 holds
    z[0, 2, int(ids[0, 2, 0])] = 90.0
    check_distill(z, ids, values, lse, 1.0)


def test_distill_gradient_against_differences():
    """The kernel's gradient against central differences of the plain loss: its third-order term is below 2e-8
    at a step of 1e-3 (|d3 loss| <= tau^2 / tau^3 per unit), the 64-bit loss' rounding below 1e-12."""
    z = rows(1, 2, 40, torch.float32, 31, scale=1.0)
    for tail in (False, True):
        ids, values, lse = teacher(z, 6, 1.5, tail, 2)
        got = dca.distill(z, ids.cuda(), values.cuda(), None if lse is None else lse.cuda(), temperature=1.5,
                          grad_loss=torch.ones((1, 2), device="cuda"))["grad"].cpu().numpy()
        x, step = host(z).astype(np.float64), 1e-3
        for r in range(2):
            for v in range(0, 40, 3):
                d = []
                for sign in (1, -1):
                    w = x.copy()
                    w[0, r, v] += sign * step
                    d.append(plain.distill(w, ids.numpy(), values.numpy(), None if lse is None else lse.numpy(),
                                           1.5)[0][0, r])
                assert abs((d[0] - d[1]) / (2 * step) - got[0, r, v]) <= 1e-6 + 2 * SUM, (tail, r, v)


def test_distill_gradient_rows_of_other_strides():
    z = rows(2, 3, 3001, torch.bfloat16, 9, pad=5, shift=1)
    ids, values, lse = teacher(z, 12, 1.0, True, 3)
    g = torch.ones((2, 3), device="cuda")
    args = dict(ids=ids.cuda(), values=values.cuda(), teacher_lse=lse.cuda(), grad_loss=g)
    want = dca.distill(z, **args)["grad"]
    room = torch.full((2, 4, 3010), 7.0, dtype=torch.bfloat16, device="cuda")
    got = dca.distill(z, out={"grad": room[:, :3, 2:3003]}, **args)["grad"]
    assert torch.equal(got.contiguous(), want)
    rest = room.clone()
    rest[:, :3, 2:3003] = 7.0
    assert (rest == 7.0).all()  # nothing written beside the rows


# ---- streams and graphs ----

def test_operators_on_a_stream_of_their_own():
    z = rows(4, 6, 30011, torch.float32, 77)
    want = dca.top_logits(z, 16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = dca.top_logits(z, 16)
        d = dca.distill(z, got["ids"], got["values"], got["lse"], grad_loss=torch.ones((4, 6), device="cuda"))
    torch.cuda.current_stream().wait_stream(side)
    for name in want:
        assert torch.equal(want[name], got[name]), name
    # a student that is its own teacher: the masses are equal, the loss is 0 within the bound
    assert float(d["loss"].abs().max()) <= 2 * SUM + 20 * H


def test_operators_replayed_from_a_graph():
    B, W, V, k = 3, 4, 20011, 12
    z = rows(B, W, V, torch.float32, 1)
    scores, state = some_scores(B, W, 1).cuda(), torch.randn((B, W, 64), device="cuda")
    g = torch.ones((B, W), device="cuda")

    def step():
        t = dca.top_logits(z, k)
        b = dca.beam_step(z, scores, n_out=6, state=state)
        d = dca.distill(z, t["ids"], t["values"], t["lse"], temperature=2.0, grad_loss=g)
        return {**{"t_" + n: x for n, x in t.items()}, **{"b_" + n: x for n, x in b.items()},
                **{"d_" + n: x for n, x in d.items()}}

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for seed in range(2, 6):
        z.copy_(rows(B, W, V, torch.float32, seed))
        scores.copy_(some_scores(B, W, seed))
        graph.replay()
        torch.cuda.synchronize()
        want = step()
        torch.cuda.synchronize()
        for name in want:
            assert torch.equal(held[name].view(torch.uint8), want[name].view(torch.uint8)), (seed, name)


# ---- refusals of the Python functions (nothing is launched) ----

def test_python_functions_refuse_mistyped_tensors():
    z = rows(2, 3, 50, torch.float32, 1)
    ids, values = (t.cuda() for t in teacher(z, 4, 1.0, False, 1)[:2])
    scores, g = some_scores(2, 3, 1).cuda(), torch.ones((2, 3), device="cuda")
    half = torch.zeros((2, 3, 50), dtype=torch.float16, device="cuda")
    bad = [
        lambda: dca.top_logits(half, 4), lambda: dca.top_logits(z.transpose(1, 2), 2),
        lambda: dca.top_logits(z[0, 0], 4), lambda: dca.top_logits(z, 4, n_rows=torch.ones(2, device="cuda")),
        lambda: dca.top_logits(z, 4, out={"ids": torch.empty((2, 3, 4), device="cuda")}),
        lambda: dca.top_logits(z, 4, out={"tokens": ids}), lambda: dca.top_logits(z, 4, workspace=g),
        lambda: dca.beam_step(z[0], scores[:1]), lambda: dca.beam_step(z, scores.double()),
        lambda: dca.beam_step(z, scores[:, :2]), lambda: dca.beam_step(z, scores.cpu()),
        lambda: dca.beam_step(z, scores, eos=1, finished=ids[..., 0]),
        lambda: dca.beam_step(z, scores, state=scores[:1]), lambda: dca.beam_step(z, scores, state=g, out={"state": g}),
        lambda: dca.beam_step(z, scores, history=ids.long()), lambda: dca.beam_step(z, scores, out={"scores": scores}),
        lambda: dca.distill(z, ids.long(), values), lambda: dca.distill(z, ids, values[..., :3]),
        lambda: dca.distill(z, ids[:1], values), lambda: dca.distill(z, ids, values, teacher_lse=g[:1]),
        lambda: dca.distill(z, ids, values, grad_loss=g, out={"grad": half}),
        lambda: dca.distill(z, ids, values, out={"grad": z}),
        lambda: dca.distill_backward(z, ids, torch.zeros((2, 3, 7), device="cuda"), g),
        lambda: dca.distill_backward(z, ids, torch.zeros((2, 3, 8), device="cuda"), g, out=z[:1]),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail("call %d was not refused" % i)
    with pytest.raises(dca.DominoError, match="EINVAL"):
        dca.top_logits(z, 51)
    with pytest.raises(dca.DominoError, match="EINVAL"):
        dca.beam_step(z, scores, finished=torch.zeros((2, 3), dtype=torch.bool, device="cuda"))  # no eos
    with pytest.raises(dca.DominoError, match="EWORKSPACE"):
        dca.top_logits(rows(1, 1, 40000, torch.float32, 1), 4,
                       workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
