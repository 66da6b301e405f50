"""Measured cases of the operators that train a head on given tokens: token log-probabilities, linear layers, embedding.

Each operator has a plain form (elementary torch operations) and the framework's entry point; `own` says which of the
two `run` takes.

* score:  log-probabilities of given tokens under rows of logits [B, R, V], with the entropy of the rows and the k most
          likely alternatives (mode "score"); forward, then the logits' gradient from the rows' statistics (mode "two");
          both in one call (mode "both").  A token outside [0, V) leaves its row out, as rows past n_rows are.
* linear: y = act(x w^T + bias) + residual over M rows, with what the backward pass needs of it (mode "forward"); the
          gradients of x, w and bias (mode "backward").
* embed:  rows of a table by token, scaled (mode "forward"); the table's gradient, summed token by token (mode
          "backward").
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # the smallest head's vocabulary: nothing but latency
        dict(name="score_tiny", op="score", mode="score", B=2, R=16, V=1024, pad=0, dtype="f32", k=4, tau=1.0,
             ragged=False),
        # a serving batch of 32 blocks whose tokens are reported with their 20 likeliest alternatives
        dict(name="score_report_batch32", op="score", mode="score", B=32, R=16, V=151936, pad=0, dtype="bf16", k=20,
             tau=1.0, ragged=False),
        # a policy step on the same rows: advantages are known after the forward pass, entropy is rewarded
        dict(name="score_two_calls", op="score", mode="two", B=32, R=16, V=151936, pad=0, dtype="bf16", k=0, tau=1.0,
             ragged=False),
        # accepted prefixes of different lengths, ignored tokens, an odd vocabulary; loss and gradient together
        dict(name="score_both_ragged_odd", op="score", mode="both", B=48, R=16, V=50021, pad=3, dtype="f32", k=0,
             tau=0.7, ragged=True),
        # the corrected logits of one block: u in float32, W2 in bfloat16, base logits added
        dict(name="linear_one_block", op="linear", mode="forward", M=16, K=256, N=151936, x="f32", w="bf16", y="f32",
             bias=False, act="", residual="f32", pre=False),
        # the low-rank layer of a batch of 32 blocks: long rows, few outputs, its pre-activation kept for training
        dict(name="linear_low_rank", op="linear", mode="forward", M=512, K=5120, N=256, x="bf16", w="bf16", y="bf16",
             bias=False, act="silu", residual="", pre=True),
        # the corrected logits of the same batch
        dict(name="linear_logits_batch32", op="linear", mode="forward", M=512, K=256, N=151936, x="bf16", w="bf16",
             y="f32", bias=False, act="", residual="f32", pre=False),
        # gradients of the same layer: sums over the vocabulary, and over the rows
        dict(name="linear_back_batch32", op="linear", mode="backward", M=512, K=256, N=151936, g="bf16", x="bf16",
             w="bf16", dx="bf16", dw="f32", bias=False, act=""),
        # a small layer of odd sizes in float32, all gradients
        dict(name="linear_back_odd", op="linear", mode="backward", M=331, K=1091, N=203, g="f32", x="f32", w="f32",
             dx="f32", dw="f32", bias=True, act="gelu"),
        # embeddings of the drafted tokens of 256 blocks
        dict(name="embed_batch256", op="embed", mode="forward", T=4096, V=151936, d=4096, table="bf16", out="bf16",
             scale=1.0, spread="zipf"),
        # the gradient of the smallest head's table: nothing but latency
        dict(name="embed_back_tiny", op="embed", mode="backward", T=32, V=1024, d=64, grad="f32", table="f32", scale=1.0,
             spread="even"),
        # the gradient of a table of states, for 256 blocks: most rows of the vocabulary are not among the tokens
        dict(name="embed_back_batch256", op="embed", mode="backward", T=4096, V=151936, d=1024, grad="f32", table="f32",
             scale=0.5, spread="zipf"),
    ]


def draw(rng):
    def log_int(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    def pick(*names):
        return rng.choice(names)

    op = pick("score", "linear", "linear", "embed")
    if op == "score":
        mode = pick("score", "score", "two", "both")
        V = log_int(1000, 151936)
        return dict(op=op, mode=mode, B=log_int(1, 32), R=rng.randint(1, 16), V=V, pad=pick(0, 0, 1, 8, 61),
                    dtype=pick("f32", "bf16"), k=pick(0, log_int(1, 128)) if mode == "score" else 0,
                    tau=pick(0.7, 1.0, 2.0), ragged=rng.random() < 0.4)
    if op == "linear":
        mode = pick("forward", "backward")
        M = log_int(1, 512)
        # one long side at the most: the vocabulary, or the width that a layer reads
        N, K = (log_int(1000, 151936), log_int(16, 256)) if rng.random() < 0.5 else (log_int(16, 1024), log_int(64, 5120))
        case = dict(op=op, mode=mode, M=M, K=K, N=N, x=pick("f32", "bf16"), w=pick("f32", "bf16"),
                    bias=rng.random() < 0.5, act=pick("", "", "silu", "gelu", "relu"))
        if mode == "forward":
            case.update(y=pick("f32", "bf16"), residual=pick("", "f32", "bf16"), pre=rng.random() < 0.3)
        else:
            case.update(g=pick("f32", "bf16"), dx=pick("f32", "bf16"), dw=pick("f32", "bf16"))
        return case
    case = dict(op=op, mode=pick("forward", "backward"), T=log_int(1, 4096), V=log_int(1000, 151936),
                d=log_int(48, 1024), table=pick("f32", "bf16"), scale=pick(1.0, 0.5, 8.0),
                spread=pick("zipf", "even", "one"))
    case["out" if case["mode"] == "forward" else "grad"] = pick("f32", "bf16")
    return case


def _lengths(case):
    """Rows of each block that count, of R: any length from none to all."""
    R = case["R"]
    return [(7 * b + 3) % (R + 1) for b in range(case["B"])] if case["ragged"] else [R] * case["B"]


def _prepare_score(case, g):
    dev = {"device": "cuda"}
    B, R, V, k = case["B"], case["R"], case["V"], case["k"]
    wide = torch.empty((B, R, V + case["pad"]), dtype=DTYPES[case["dtype"]], **dev)
    tokens = torch.empty((B, R), dtype=torch.int32, **dev)
    for b in range(B):  # broad noise, a few tokens well above it, another sharpness in each row
        x = 2.5 * torch.randn((R, V + case["pad"]), generator=g, **dev)
        peak = torch.randint(0, V, (R, 6), generator=g, **dev)
        x.scatter_(1, peak, 12.0 - 1.5 * torch.arange(6, **dev).float().expand(R, 6)
                   + torch.randn((R, 6), generator=g, **dev))
        wide[b] = x * (0.6 + torch.rand((R, 1), generator=g, **dev))
        # mostly one of the likely tokens, else any
        at = torch.randint(0, 6, (R, 1), generator=g, **dev)
        rare = torch.randint(0, V, (R,), generator=g, **dev)
        tokens[b] = torch.where(torch.rand(R, generator=g, **dev) < 0.9, peak.gather(1, at)[:, 0], rare).int()
    if case["ragged"]:
        tokens.view(-1)[4::11] = -1
    state = dict(case=case, logits=wide[..., :V], tokens=tokens,
                 n_rows=torch.tensor(_lengths(case), dtype=torch.int32, **dev) if case["ragged"] else None)
    out = {"logprob": torch.empty((B, R), **dev), "entropy": torch.empty((B, R), **dev)}
    if k:
        out.update(ids=torch.empty((B, R, k), dtype=torch.int32, **dev), logprobs=torch.empty((B, R, k), **dev))
    if case["mode"] != "score":
        state["grad_logprob"] = torch.randn((B, R), generator=g, **dev) / (B * R)
        state["grad_entropy"] = torch.full((B, R), 0.01 / (B * R), **dev)
        out["grad"] = torch.empty((B, R, V), dtype=DTYPES[case["dtype"]], **dev)
    state["out"] = out
    return state


def _prepare_linear(case, g):
    M, K, N, dev = case["M"], case["K"], case["N"], {"device": "cuda"}

    def normal(*shape):
        return torch.randn(shape, generator=g, **dev)

    x = normal(M, K)
    state = dict(case=case, x=(x * torch.sigmoid(x)).to(DTYPES[case["x"]]),
                 w=(normal(N, K) / math.sqrt(K)).to(DTYPES[case["w"]]))
    if case["mode"] == "forward":
        state["bias"] = normal(N) if case["bias"] else None
        state["residual"] = (3.0 * normal(M, N)).to(DTYPES[case["residual"]]) if case["residual"] else None
        state["out"] = {"y": torch.empty((M, N), dtype=DTYPES[case["y"]], **dev)}
        if case["pre"]:
            state["out"]["pre"] = torch.empty((M, N), **dev)
        return state
    # the gradient of a likelihood: each row a distribution less its token, weighted
    p = torch.softmax(2.0 * normal(M, N), 1)
    p[torch.arange(M, **dev), torch.randint(0, N, (M,), generator=g, **dev)] -= 1.0
    state["grad"] = (p * (0.5 + torch.rand((M, 1), generator=g, **dev)) / M).to(DTYPES[case["g"]])
    state["pre"] = normal(M, N) if case["act"] else None
    state["out"] = {"x": torch.empty((M, K), dtype=DTYPES[case["dx"]], **dev),
                    "weight": torch.empty((N, K), dtype=DTYPES[case["dw"]], **dev)}
    if case["bias"]:
        state["out"]["bias"] = torch.empty(N, **dev)
    return state


def _prepare_embed(case, g):
    T, V, d, dev = case["T"], case["V"], case["d"], {"device": "cuda"}
    if case["spread"] == "one":  # one token, as padding gives
        ids = torch.full((T,), int(torch.randint(0, V, (1,), generator=g, **dev)), dtype=torch.int32, **dev)
    elif case["spread"] == "zipf":  # the frequency of rank r falls as 1 / r
        ids = torch.exp(torch.rand(T, generator=g, **dev).double() * math.log(V)).long().clamp(1, V).sub(1).int()
    else:
        ids = torch.randint(0, V, (T,), generator=g, dtype=torch.int32, **dev)
    state = dict(case=case, ids=ids)
    if case["mode"] == "forward":
        state["table"] = (0.02 * torch.randn((V, d), generator=g, **dev)).to(DTYPES[case["table"]])
        state["out"] = torch.empty((T, d), dtype=DTYPES[case["out"]], **dev)
    else:
        state["grad"] = (0.01 * torch.randn((T, d), generator=g, **dev)).to(DTYPES[case["grad"]])
        state["out"] = torch.empty((V, d), dtype=DTYPES[case["table"]], **dev)
    return state


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return {"score": _prepare_score, "linear": _prepare_linear, "embed": _prepare_embed}[case["op"]](case, g)


def run(state):
    case = state["case"]
    if own:
        import causal_draft_correction_amd as dca

        if case["op"] == "embed":
            if case["mode"] == "forward":
                return dca.embed(state["table"], state["ids"], scale=case["scale"], out=state["out"])
            return dca.embed_backward(state["grad"], state["ids"], case["V"], scale=case["scale"], out=state["out"])
        if case["op"] == "linear":
            if case["mode"] == "forward":
                return dca.linear(state["x"], state["w"], bias=state["bias"], activation=case["act"] or None,
                                  residual=state["residual"], want_pre=case["pre"], out=state["out"])
            return dca.linear_backward(state["grad"], state["x"], state["w"], pre=state["pre"],
                                       activation=case["act"] or None, want=tuple(state["out"]), out=state["out"])
        rows = dict(temperature=case["tau"], n_rows=state["n_rows"])
        if case["mode"] == "score":
            return dca.token_logprobs(state["logits"], state["tokens"], k=case["k"], out=state["out"], **rows)
        if case["mode"] == "both":
            return dca.token_logprobs(state["logits"], state["tokens"], grad_logprob=state["grad_logprob"],
                                      grad_entropy=state["grad_entropy"], out=state["out"], **rows)
        got = dca.token_logprobs(state["logits"], state["tokens"], want_stats=True,
                                 out={name: state["out"][name] for name in ("logprob", "entropy")}, **rows)
        grad = dca.token_logprobs_backward(state["logits"], state["tokens"], got["stats"], state["grad_logprob"],
                                           grad_entropy=state["grad_entropy"], out=state["out"]["grad"], **rows)
        return {"logprob": got["logprob"], "entropy": got["entropy"], "grad": grad}
    return {"score": _plain_score, "linear": _plain_linear, "embed": _plain_embed}[case["op"]](state)


def _largest(x, k):
    """Indices of the k largest of each row, largest first, ties to the lowest index."""
    bits = (x + 0.0).view(torch.int32)
    order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long()
    V = x.shape[-1]
    keys = (order << 32) + (V - 1 - torch.arange(V, device=x.device))
    return V - 1 - (keys.topk(k).values & 0xFFFFFFFF)


def _plain_score(state):
    case, V, tau = state["case"], state["case"]["V"], state["case"]["tau"]
    B, R = case["B"], case["R"]
    x, token = state["logits"].float(), state["tokens"].long()
    live = (token >= 0) & (token < V)
    if state["n_rows"] is not None:
        live = live & (torch.arange(R, device="cuda") < state["n_rows"][:, None])
    m = x.amax(-1, keepdim=True)
    d = (x - m) / tau
    e = torch.exp(d)
    # few values a row in 64 bits: a logarithm of nearly 1, and differences of logarithms
    total = e.sum(-1)
    log_total = torch.log(e.double().sum(-1))
    entropy = log_total - (e * d).sum(-1).double() / total.double()
    token = token.clamp(0, V - 1)[..., None]
    logprob = d.gather(-1, token)[..., 0].double() - log_total
    out = {"logprob": torch.where(live, logprob, 0.0).float(), "entropy": torch.where(live, entropy, 0.0).float()}
    if case["k"]:
        ids = _largest(x, case["k"])
        logprobs = d.gather(-1, ids).double() - log_total[..., None]
        out["ids"] = torch.where(live[..., None], ids, -1).int()
        out["logprobs"] = torch.where(live[..., None], logprobs, -math.inf).float()
    if case["mode"] == "score":
        return out
    # dlogprob/dz = (1[v is the token] - p) / tau, dentropy/dz = -p (log p + entropy) / tau
    glp, gh = state["grad_logprob"][..., None], state["grad_entropy"][..., None]
    p = e / total[..., None]
    grad = -p * (glp + gh * (d + (entropy - log_total).float()[..., None]))
    grad = grad.scatter_add(-1, token, glp.expand(B, R, 1)) / tau
    out["grad"] = torch.where(live[..., None], grad, 0.0).to(state["logits"].dtype)
    return out


def _act(a, name):
    if name == "silu":
        return a * torch.sigmoid(a)
    if name == "gelu":
        return 0.5 * a * torch.erfc(-a * math.sqrt(0.5))
    return a.clamp(min=0) if name == "relu" else a


def _slope(a, name):
    if name == "silu":
        s = torch.sigmoid(a)
        return s * (1.0 + a * (1.0 - s))
    if name == "gelu":
        return 0.5 * torch.erfc(-a * math.sqrt(0.5)) + a * torch.exp(-0.5 * a * a) / math.sqrt(2.0 * math.pi)
    return (a > 0).float()


def _plain_linear(state):
    case, x, w = state["case"], state["x"].float(), state["w"].float()
    if case["mode"] == "forward":
        pre = x @ w.t()
        if case["bias"]:
            pre = pre + state["bias"]
        y = _act(pre, case["act"])
        if case["residual"]:
            y = y + state["residual"].float()
        return {"y": y.to(DTYPES[case["y"]]), "pre": pre} if case["pre"] else {"y": y.to(DTYPES[case["y"]])}
    g = state["grad"].float()
    if case["act"]:
        g = g * _slope(state["pre"], case["act"])
    out = {"x": (g @ w).to(DTYPES[case["dx"]]), "weight": (g.t() @ x).to(DTYPES[case["dw"]])}
    if case["bias"]:
        out["bias"] = g.sum(0)
    return out


def _plain_embed(state):
    case, ids = state["case"], state["ids"].long()
    if case["mode"] == "forward":
        return (state["table"][ids].float() * case["scale"]).to(DTYPES[case["out"]])
    total = torch.zeros((case["V"], case["d"]), device="cuda")
    total.index_add_(0, ids, state["grad"].float())
    return (total * case["scale"]).to(DTYPES[case["table"]])


def exact(case, seed):
    """The definitions in 64 bits: softmax over whole rows with its gradients by differentiation, dense products with
    theirs, one product with the tokens' indicator matrix for the table's gradient."""
    state = prepare(case, seed)
    if case["op"] == "embed":
        if case["mode"] == "forward":
            return torch.index_select(state["table"], 0, state["ids"]).double().mul(case["scale"])
        used, where = torch.unique(state["ids"], return_inverse=True)
        hot = torch.zeros((len(used), case["T"]), dtype=torch.float64, device="cuda")
        hot[where, torch.arange(case["T"], device="cuda")] = case["scale"]
        full = torch.zeros((case["V"], case["d"]), dtype=torch.float64, device="cuda")
        full[used.long()] = hot @ state["grad"].double()
        return full
    if case["op"] == "linear":
        acts = {"": lambda a: a, "silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu, "relu": torch.relu}
        x, w = state["x"].double(), state["w"].double()
        if case["mode"] == "forward":
            pre = torch.nn.functional.linear(x, w, None if state["bias"] is None else state["bias"].double())
            y = acts[case["act"]](pre)
            y = y if state["residual"] is None else y + state["residual"]
            return {"y": y, "pre": pre} if case["pre"] else {"y": y}
        g = state["grad"].double()
        if case["act"]:
            pre = state["pre"].double().requires_grad_()
            g, = torch.autograd.grad(acts[case["act"]](pre), pre, g)
        out = {"x": torch.mm(g, w), "weight": torch.mm(g.t(), x)}
        if case["bias"]:
            out["bias"] = torch.mv(g.t(), torch.ones(case["M"], dtype=torch.float64, device="cuda"))
        return out
    V, tau = case["V"], case["tau"]
    out = {"logprob": [], "entropy": [], "logprobs": [], "grad": []}
    lengths = _lengths(case)
    for b in range(case["B"]):  # (block by block: the rows are held several times over)
        z = state["logits"][b].double().requires_grad_(case["mode"] != "score")
        token = state["tokens"][b].long()
        live = (token >= 0) & (token < V) & (torch.arange(case["R"], device="cuda") < lengths[b])
        logp = torch.log_softmax(z / tau, -1)
        logprob = logp.gather(-1, token.clamp(0, V - 1)[:, None])[:, 0] * live
        entropy = torch.special.entr(logp.exp()).sum(-1) * live
        out["logprob"].append(logprob.detach())
        out["entropy"].append(entropy.detach())
        if case["k"]:
            best = logp.sort(dim=-1, descending=True).values[:, :case["k"]]
            out["logprobs"].append(best.masked_fill(~live[:, None], -math.inf))
        if case["mode"] != "score":
            value = (logprob * state["grad_logprob"][b].double()).sum() + (entropy * state["grad_entropy"][b].double()).sum()
            grad, = torch.autograd.grad(value, z)
            out["grad"].append(grad)
    out = {name: torch.stack(rows) for name, rows in out.items() if rows}
    if case["k"]:
        out["ids"] = None
    return out


def work(case):
    size = {"f32": 4, "bf16": 2, "": 0}
    if case["op"] == "embed":
        T, V, d = case["T"], case["V"], case["d"]
        if case["mode"] == "forward":
            return {"bytes": T * (4 + d * (size[case["table"]] + size[case["out"]])), "flops": T * d}
        return {"bytes": T * (4 + d * size[case["grad"]]) + V * d * size[case["table"]], "flops": T * d}
    if case["op"] == "linear":
        M, K, N = case["M"], case["K"], case["N"]
        own_bytes = M * K * size[case["x"]] + N * K * size[case["w"]] + 4 * N * case["bias"]
        if case["mode"] == "forward":
            return {"bytes": own_bytes + M * N * (size[case["y"]] + size[case["residual"]] + 4 * case["pre"]),
                    "flops": 2 * M * N * K}
        return {"bytes": own_bytes + M * N * (size[case["g"]] + (4 if case["act"] else 0)) + M * K * size[case["dx"]] +
                N * K * size[case["dw"]], "flops": 4 * M * N * K}
    s, rows = size[case["dtype"]], sum(_lengths(case))
    n, every = rows * case["V"], case["B"] * case["R"]
    small = every * (12 + 8 * case["k"])
    if case["mode"] == "score":
        return {"bytes": n * s + small, "flops": 6 * n}
    return {"bytes": n * s + every * case["V"] * s + small + 8 * every, "flops": 11 * n}
