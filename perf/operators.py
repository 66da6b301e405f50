"""Measured cases of the operators over vocabulary rows: top logits, beam selection, distillation.

Each operator has a plain form (elementary torch operations) and the framework's entry point; `own`
says which of the two `run` takes.  Rows of logits are [B, R, V] views whose last dimension is
contiguous; `pad` columns may follow each row, as in a vocabulary padded to a round width.

* top:     the k largest logits of each row (largest first, ties to the lowest id), with their ids and
           the log-sum-exp of the row at temperature tau: what a teacher leaves behind for distillation.
* beam:    one step of beam search: the M best continuations of W beams over the vocabulary, with the
           beams' recurrent state and token history put in the new order.
* distill: the loss of a student's logits against a teacher's top logits at temperature tau, per row,
           and its gradient (mode "loss": forward alone; "two": forward, then backward; "both": loss
           and gradient in one call).
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
EOS = 2


def listed():
    return [
        # the target's logits of one verified block of 16 drafted tokens, kept as 64 teacher logits a row
        dict(name="top_one_block", op="top", B=1, R=17, V=151936, pad=0, dtype="f32", k=64, tau=1.0, ragged=False),
        # the same for a serving batch of 32 blocks whose logits stay in bfloat16
        dict(name="top_batch32", op="top", B=32, R=16, V=151936, pad=0, dtype="bf16", k=20, tau=1.0, ragged=False),
        # the smallest head's vocabulary: nothing but latency
        dict(name="top_tiny", op="top", B=2, R=16, V=1024, pad=0, dtype="f32", k=8, tau=1.0, ragged=False),
        # accepted prefixes of different lengths, an odd vocabulary: rows begin at any address
        dict(name="top_ragged_odd", op="top", B=24, R=16, V=50021, pad=0, dtype="bf16", k=33, tau=2.0, ragged=True),
        # the first step of a small head's beam search: one live beam
        dict(name="beam_tiny_first", op="beam", B=1, W=4, V=1024, pad=0, dtype="f32", M=4, h=64, T=16, step=0,
             dead=3, ended=0),
        # drafting one block with four beams: latency of one position
        dict(name="beam_one_request", op="beam", B=1, W=4, V=151936, pad=0, dtype="f32", M=8, h=1024, T=16, step=3,
             dead=0, ended=0),
        # a serving batch with one ended beam in each request
        dict(name="beam_batch32", op="beam", B=32, W=8, V=151936, pad=0, dtype="bf16", M=16, h=1024, T=16, step=7,
             dead=0, ended=1),
        # a padded odd vocabulary and an uneven number of continuations
        dict(name="beam_padded_odd", op="beam", B=16, W=7, V=32003, pad=61, dtype="f32", M=13, h=256, T=12, step=11,
             dead=1, ended=1),
        # training the smallest head: nothing but latency
        dict(name="distill_tiny", op="distill", mode="both", B=2, R=16, V=1024, pad=0, dtype="f32", k=8, tau=1.0,
             tail=True, ragged=False),
        # the loss alone, as an evaluation reports it, over accepted prefixes of different lengths
        dict(name="distill_loss_ragged", op="distill", mode="loss", B=16, R=16, V=151936, pad=0, dtype="f32", k=64,
             tau=1.0, tail=True, ragged=True),
        # a training step whose loss is weighted after the forward pass: forward, then backward
        dict(name="distill_two_calls", op="distill", mode="two", B=32, R=16, V=151936, pad=0, dtype="bf16", k=32,
             tau=2.0, tail=False, ragged=False),
        # the largest training step: 64 blocks of 16 positions, loss and gradient together
        dict(name="distill_batch64", op="distill", mode="both", B=64, R=16, V=151936, pad=0, dtype="f32", k=64,
             tau=1.0, tail=True, ragged=False),
    ]


def draw(rng):
    def log_int(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["top", "beam", "distill", "distill"])
    case = dict(op=op, V=log_int(1000, 151936), pad=rng.choice([0, 0, 1, 8, 61]), dtype=rng.choice(["f32", "bf16"]))
    if op == "beam":
        W = rng.randint(2, 16)
        case.update(B=log_int(1, 48), W=W, M=rng.randint(W, 2 * W), h=rng.choice([64, 200, 512, 1024]),
                    T=16, step=rng.randint(0, 15), dead=rng.choice([0, 0, 1, W - 1]), ended=0)
        if case["dead"] < W - 1:
            case["ended"] = rng.choice([0, 1])
        return case
    case.update(B=log_int(1, 64), R=rng.randint(1, 16), k=log_int(1, 128), tau=rng.choice([0.7, 1.0, 2.0]),
                ragged=rng.random() < 0.4)
    if op == "distill":
        case.update(mode=rng.choice(["loss", "two", "both"]), tail=rng.random() < 0.6)
    return case


def _lengths(case):
    """Rows of each block that count, of R: any length from none to all."""
    R = case["R"]
    return [(7 * b + 3) % (R + 1) for b in range(case["B"])] if case["ragged"] else [R] * case["B"]


def _logits(g, case, rows):
    """Rows as a model gives them: broad noise, a few tokens well above it, another sharpness in each row."""
    B, V = case["B"], case["V"]
    wide = torch.empty((B, rows, V + case["pad"]), device="cuda", dtype=DTYPES[case["dtype"]])
    for b in range(B):
        x = 2.5 * torch.randn((rows, V + case["pad"]), device="cuda", generator=g)
        n = 6
        peak = torch.randint(0, V, (rows, n), device="cuda", generator=g)
        x.scatter_(1, peak, 12.0 - 1.5 * torch.arange(n, device="cuda").float().expand(rows, n)
                   + torch.randn((rows, n), device="cuda", generator=g))
        wide[b] = x * (0.6 + torch.rand((rows, 1), device="cuda", generator=g))
    return wide[..., :V]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = {"device": "cuda"}
    B, V, op = case["B"], case["V"], case["op"]
    if op == "beam":
        W, M, T = case["W"], case["M"], case["T"]
        logits = _logits(g, case, W)
        scores = -torch.cumsum(0.2 + 1.5 * torch.rand((B, W), generator=g, **dev), 1)
        finished = torch.zeros((B, W), dtype=torch.bool, **dev)
        if case["dead"]:
            scores[:, W - case["dead"]:] = -math.inf
        if case["ended"]:
            finished[:, 1:1 + case["ended"]] = True
        # unused places hold 0, tokens already chosen lie before `step`
        history = torch.randint(0, V, (B, W, T), generator=g, dtype=torch.int32, **dev)
        history[:, :, case["step"]:] = 0
        out = {"scores": torch.empty((B, M), **dev), "parent": torch.empty((B, M), dtype=torch.int32, **dev),
               "token": torch.empty((B, M), dtype=torch.int32, **dev),
               "finished": torch.empty((B, M), dtype=torch.bool, **dev), "state": torch.empty((B, M, case["h"]), **dev),
               "history": torch.empty((B, M, T), dtype=torch.int32, **dev)}
        return dict(case=case, logits=logits, scores=scores, finished=finished, history=history, out=out,
                    state=torch.tanh(torch.randn((B, W, case["h"]), generator=g, **dev)))
    R, k, tau = case["R"], case["k"], case["tau"]
    logits = _logits(g, case, R)
    n_rows = torch.tensor(_lengths(case), dtype=torch.int32, **dev) if case["ragged"] else None
    if op == "top":
        out = {"ids": torch.empty((B, R, k), dtype=torch.int32, **dev), "values": torch.empty((B, R, k), **dev),
               "lse": torch.empty((B, R), **dev)}
        return dict(case=case, logits=logits, n_rows=n_rows, out=out)
    ids = torch.empty((B, R, k), dtype=torch.int32, **dev)
    values = torch.empty((B, R, k), **dev)
    lse = torch.empty((B, R), **dev)
    for b in range(B):  # a teacher that agrees with the student in the main
        t = logits[b].float() + 0.8 * torch.randn((R, V), generator=g, **dev)
        v, i = t.topk(k)
        ids[b], values[b], lse[b] = i.int(), v, torch.logsumexp(t / tau, 1)
    out = {"loss": torch.empty((B, R), **dev)}
    state = dict(case=case, logits=logits, n_rows=n_rows, ids=ids, values=values,
                 teacher_lse=lse if case["tail"] else None, out=out)
    if case["mode"] != "loss":
        # later positions of a block weigh less; the mean over the batch
        weight = 0.9 ** torch.arange(R, **dev).float() / (B * R)
        state["grad_loss"] = (weight * (0.75 + 0.5 * torch.rand((B, R), generator=g, **dev))).contiguous()
        out["grad"] = torch.empty((B, R, V), dtype=DTYPES[case["dtype"]], **dev)
    return state


def run(state):
    case = state["case"]
    if own:
        import causal_draft_correction_amd as dca

        if case["op"] == "top":
            return dca.top_logits(state["logits"], case["k"], temperature=case["tau"], n_rows=state["n_rows"],
                                  out=state["out"])
        if case["op"] == "beam":
            return dca.beam_step(state["logits"], state["scores"], n_out=case["M"], eos=EOS,
                                 finished=state["finished"], state=state["state"], history=state["history"],
                                 step=case["step"], out=state["out"])
        teacher = dict(teacher_lse=state["teacher_lse"], temperature=case["tau"], n_rows=state["n_rows"])
        if case["mode"] == "loss":
            return {"loss": dca.distill(state["logits"], state["ids"], state["values"], out=state["out"],
                                        **teacher)["loss"]}
        if case["mode"] == "both":
            got = dca.distill(state["logits"], state["ids"], state["values"], grad_loss=state["grad_loss"],
                              out=state["out"], **teacher)
            return {"loss": got["loss"], "grad": got["grad"]}
        got = dca.distill(state["logits"], state["ids"], state["values"], out={"loss": state["out"]["loss"]}, **teacher)
        grad = dca.distill_backward(state["logits"], state["ids"], got["stats"], state["grad_loss"],
                                    temperature=case["tau"], n_rows=state["n_rows"], out=state["out"]["grad"])
        return {"loss": got["loss"], "grad": grad}
    if case["op"] == "top":
        return _plain_top(state["logits"], case["k"], case["tau"], state["n_rows"])
    if case["op"] == "beam":
        return _plain_beam(state)
    return _plain_distill(state)


def _row_keys(x):
    """int64 keys that order a row as its float32 values do: NaN above every number, -0 as +0, ties to the
    lowest index."""
    bits = (x + 0.0).view(torch.int32)
    order = torch.where(torch.isnan(x), 0x7FFFFFFF, torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits)).long()
    V = x.shape[-1]
    return (order << 32) + (V - 1 - torch.arange(V, device=x.device))


def _largest(x, k):
    """Indices of the k largest of each row, largest first."""
    return x.shape[-1] - 1 - (_row_keys(x).topk(k).values & 0xFFFFFFFF)


def _exps(x, tau):
    """exp((x - m) / tau) with m the row's maximum, the sums of these, and the row's log-sum-exp (in 64 bits, as
    differences of logarithms are taken of it)."""
    m = x.amax(-1, keepdim=True)
    e = torch.exp((x - m) / tau)
    total = e.sum(-1)
    return e, total, m.squeeze(-1).double() / tau + torch.log(total.double())


def _counts(n_rows, B, R):
    at = torch.arange(R, device="cuda").expand(B, R)
    return at < (R if n_rows is None else n_rows[:, None])


def _plain_top(logits, k, tau, n_rows):
    x = logits.float()
    ids = _largest(x, k)
    live = _counts(n_rows, *x.shape[:2])
    none = torch.tensor(-math.inf, device="cuda")
    return {"ids": torch.where(live[..., None], ids, -1).int(),
            "values": torch.where(live[..., None], x.gather(-1, ids), none),
            "lse": torch.where(live, _exps(x, tau)[2].float(), none)}


def _plain_beam(state):
    """Scores in 64 bits: continuations of different beams lie close to each other."""
    case, scores, finished = state["case"], state["scores"].double(), state["finished"]
    B, W, V, M = case["B"], case["W"], case["V"], case["M"]
    x = state["logits"].float()
    wide = x.double()
    lse = _exps(wide, 1.0)[2]
    dead = scores == -math.inf
    bad = ~(scores < math.inf) | ~(lse < math.inf)
    cand = torch.where(x == -math.inf, -math.inf, (scores - lse)[..., None] + wide)
    cand = torch.where(bad[..., None], math.nan, cand)
    ends = torch.full((V,), -math.inf, device="cuda", dtype=torch.float64)
    ends[EOS] = 0.0
    cand = torch.where(finished[..., None], scores[..., None] + ends, cand)
    cand = torch.where(dead[..., None], -math.inf, cand)
    # the best of each beam (by its logits, which order its candidates), then of all beams
    rank = torch.where(finished[..., None], ends.float(), x)
    rank = torch.where((dead | (bad & ~finished))[..., None], 0.0, rank)
    n = min(M, V)
    token = _largest(rank, n).sort(-1).values
    best, at = cand.gather(-1, token).reshape(B, W * n).sort(dim=-1, descending=True, stable=True)
    best, at = best[:, :M], at[:, :M]
    parent, token = at // n, token.reshape(B, W * n).gather(1, at)
    T = case["T"]
    history = state["history"].gather(1, parent[..., None].expand(B, M, T))
    history[:, :, case["step"]] = token.int()
    return {"scores": best.float(), "parent": parent.int(), "token": token.int(),
            "finished": finished.gather(1, parent) | (token == EOS),
            "state": state["state"].gather(1, parent[..., None].expand(B, M, case["h"])), "history": history}


def _plain_distill(state):
    case, V, tau = state["case"], state["case"]["V"], state["case"]["tau"]
    ids, valid = state["ids"].long(), (state["ids"] >= 0) & (state["ids"] < V)
    live = _counts(state["n_rows"], case["B"], case["R"]) & valid.any(-1)
    x = state["logits"].float()
    e, total, lse = _exps(x, tau)
    # the teacher's masses: k values a row, in 64 bits (1 - their sum is small)
    t = torch.where(valid, state["values"].double() / tau, -math.inf)
    t = t - (_exps(t, 1.0)[2] if state["teacher_lse"] is None else state["teacher_lse"].double())[..., None]
    p = torch.exp(t)
    at = torch.where(valid, ids, V)
    logq = x.gather(-1, at.clamp(max=V - 1)).double() / tau - lse[..., None]
    loss = torch.where(p > 0, p * (t - logq), 0.0).sum(-1)
    rest = (1 - p.sum(-1)).clamp(min=0)
    if state["teacher_lse"] is None:
        rest = torch.zeros_like(rest)
    mass = p.sum(-1) + rest
    hit = torch.zeros((*x.shape[:2], V + 1), dtype=torch.bool, device="cuda").scatter_(-1, at, True)[..., :V]
    q_rest = torch.where(hit, 0.0, e).sum(-1).double() / total.double()
    loss = loss + torch.where(rest > 0, rest * torch.log(rest / q_rest), 0.0)
    out = {"loss": torch.where(live, tau * tau * loss, 0.0).float()}
    if case["mode"] == "loss":
        return out
    inner = torch.where(rest > 0, mass - rest / q_rest, mass)
    grad = e / total[..., None] * torch.where(hit, mass[..., None].float(), inner[..., None].float())
    grad = torch.cat([grad, torch.zeros_like(grad[..., :1])], -1).scatter_add_(-1, at, -p.float())[..., :V]
    grad = torch.where(live[..., None], grad * (tau * state["grad_loss"])[..., None], 0.0)
    out["grad"] = grad.to(state["logits"].dtype)
    return out


def exact(case, seed):
    """The definitions in 64 bits, over whole rows: a stable sort of every candidate, the loss as the divergence
    of dense distributions, its gradient by differentiation."""
    state = prepare(case, seed)
    z = state["logits"].double()
    if case["op"] == "beam":
        B, W, V, M = case["B"], case["W"], case["V"], case["M"]
        score = state["scores"].double()[..., None] + torch.log_softmax(z, -1)
        one = torch.full((V,), -math.inf, device="cuda", dtype=torch.float64)
        one[EOS] = 0.0
        score = torch.where(state["finished"][..., None], state["scores"].double()[..., None] + one, score)
        best, flat = score.reshape(B, W * V).sort(dim=1, descending=True, stable=True)
        parent = flat[:, :M] // V
        rows = torch.arange(B, device="cuda")[:, None]
        return {"scores": best[:, :M], "parent": None, "token": None, "finished": None,
                "state": state["state"].double()[rows, parent], "history": None}
    live = torch.arange(case["R"], device="cuda")[None] < torch.tensor(_lengths(case), device="cuda")[:, None]
    tau = case["tau"]
    if case["op"] == "top":
        values = z.sort(dim=-1, descending=True).values[..., :case["k"]]
        return {"ids": None, "values": values.masked_fill(~live[..., None], -math.inf),
                "lse": torch.logsumexp(z / tau, -1).masked_fill(~live, -math.inf)}
    ids, t = state["ids"].long(), state["values"].double() / tau
    logp = torch.log_softmax(t, -1) if state["teacher_lse"] is None else t - state["teacher_lse"].double()[..., None]
    z.requires_grad_(case["mode"] != "loss")
    with torch.set_grad_enabled(case["mode"] != "loss"):
        logq = torch.log_softmax(z / tau, -1)
        kl = (logp.exp() * (logp - logq.gather(-1, ids))).sum(-1)
        if state["teacher_lse"] is not None:
            other = (1 - logp.exp().sum(-1)).clamp(min=0)
            logq_other = logq.scatter(-1, ids, -math.inf).logsumexp(-1)
            kl = kl + torch.where(other > 0, torch.xlogy(other, other) - other * logq_other, 0.0)
        loss = torch.where(live, tau * tau * kl, 0.0)
    if case["mode"] == "loss":
        return {"loss": loss}
    grad, = torch.autograd.grad(loss, z, state["grad_loss"].double())
    return {"loss": loss.detach(), "grad": grad}


def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "beam":
        B, W, M = case["B"], case["W"], case["M"]
        live = B * (W - case["dead"] - case["ended"]) * case["V"]
        state = 4 * (case["h"] + case["T"])
        return {"bytes": live * size + B * W * (5 + state) + B * M * (13 + state), "flops": 3 * live}
    rows = sum(_lengths(case))
    n, all_rows = rows * case["V"], case["B"] * case["R"]
    if case["op"] == "top":
        return {"bytes": n * size + all_rows * (8 * case["k"] + 4), "flops": 4 * n}
    small = all_rows * (8 * case["k"] + 12)
    if case["mode"] == "loss":
        return {"bytes": n * size + small, "flops": 4 * n}
    return {"bytes": n * size + all_rows * case["V"] * size + small, "flops": 7 * n}
