"""Beam drafts and distillation of a Domino head: the row operators used together.

`beam_draft` drafts the W best blocks of a head instead of the greedy one: position after position the head's
corrected logits of every beam go through `beam_step`, which also puts the recurrent states in the new order.

`distill_step` is one step of adapting a head to its target: a greedy draft, the target's logits of the drafted
block, `verify`, the target's `top_logits` on the accepted prefix, `distill` of the head's logits against them, and
the gradient of W2, whose correction W2 u is what the loss reaches directly (dL/dW2 = (dL/dL_final)^T u).

    python -m causal_draft_correction_amd.adapt            # the 1024-token synthetic head
    python -m causal_draft_correction_amd.adapt qwen3_8b_b1

runs both on synthetic inputs: the target is the same head with another W2, forced on the drafted tokens.
"""
from __future__ import annotations

import sys
from typing import Callable, Optional

import torch

from .binding import DominoHead, verify
from .rows import beam_step, distill, top_logits


def beam_draft(head: DominoHead, H: torch.Tensor, L_base: torch.Tensor, last_tok: torch.Tensor, beams: int,
               eos: int = -1) -> dict:
    """The `beams` best drafts of a block for B rows, best first.

    head: a head of K = 1 positions with max_batch >= B * beams (it steps one position of every beam at a time).
    H [B, K, d], L_base [B, K, V] and last_tok [B] as `DominoHead.draft` takes them.  Returns tokens
    [B, beams, K] int32 and scores [B, beams] float32, the sums of log-probabilities.  A beam ends with `eos`
    (-1: none does) and keeps its score; its later tokens are `eos`.
    """
    B, K, V = L_base.shape
    dev = L_base.device
    if head.K != 1 or head.max_batch < B * beams:
        raise ValueError("beam_draft needs a head of K = 1 and max_batch >= %d, got K = %d and %d" %
                         (B * beams, head.K, head.max_batch))
    scores = torch.full((B, beams), -torch.inf, device=dev)
    scores[:, 0] = 0.0  # the first step has one live beam
    history = torch.zeros((B, beams, K), dtype=torch.int32, device=dev)
    finished = torch.zeros((B, beams), dtype=torch.bool, device=dev) if eos >= 0 else None
    token = last_tok.repeat_interleave(beams).contiguous()
    state = None
    for p in range(K):
        each = [x[:, p:p + 1].repeat_interleave(beams, 0) for x in (H, L_base)]
        out = head.draft(each[0], each[1], token, S_init=None if state is None else state.view(B * beams, -1),
                         want_logits=True, want_state=not head.markov)
        got = beam_step(out["L_final"].view(B, beams, V), scores, eos=eos, finished=finished,
                        state=None if head.markov else out["S"].view(B, beams, -1), history=history, step=p)
        scores, history, state, finished = got["scores"], got["history"], got.get("state"), got.get("finished")
        token = got["token"].view(-1)
    return {"tokens": history, "scores": scores}


def distill_step(weights: dict, W2: torch.Tensor, H: torch.Tensor, L_base: torch.Tensor, last_tok: torch.Tensor,
                 target: Callable[[torch.Tensor], torch.Tensor], k: int = 64, temperature: float = 1.0,
                 decay: float = 0.9) -> dict:
    """Loss of a head against its target's choices, and its gradient in W2.grad (for the caller's optimizer).

    weights: the head's weights, with W2 [V, r] float32 in the place of their own W2.  target(tokens [B, K]) gives
    the target's logits [B, K+1, V] (float32) of a drafted block.  The loss of the positions the target can judge
    (the accepted prefix and the first difference) is averaged, later ones of a block weighing decay^position.
    Returns the loss, the mean accept length and the drafted tokens.
    """
    B, K, V = L_base.shape
    # (a handle borrows its weights unchanged, so the step's W2 gets one of its own)
    head = DominoHead({**weights, "W2": W2.detach().to(weights["W2"].dtype).contiguous()}, K=K, max_batch=B)
    out = head.draft(H, L_base, last_tok, want_logits=True, want_state=True)
    logits = target(out["tokens"])
    checked = verify(logits, out["tokens"])
    judged = (checked["accept"] + 1).clamp_(max=K)
    teacher = top_logits(logits[:, :K], k, temperature=temperature, n_rows=judged)
    weight = (decay ** torch.arange(K, device=W2.device)).expand(B, K) * \
        (torch.arange(K, device=W2.device) < judged[:, None])
    weight = (weight / weight.sum()).contiguous()
    # the gradient takes the place of the logits
    got = distill(out["L_final"], teacher["ids"], teacher["values"], teacher["lse"], temperature=temperature,
                  n_rows=judged, grad_loss=weight, out={"grad": out["L_final"]})
    W2.grad = got["grad"].view(B * K, V).t() @ out["u"].view(B * K, -1)
    return {"loss": (got["loss"] * weight).sum(), "accept": checked["accept"].float().mean(), "tokens": out["tokens"]}


def synthetic_target(weights: dict, W2: torch.Tensor, H: torch.Tensor, L_base: torch.Tensor,
                     last_tok: torch.Tensor) -> Callable[[torch.Tensor], torch.Tensor]:
    """A target that is the head itself with another W2, forced on the drafted tokens; its last row, which follows
    the whole block, is the block's last base logits."""
    B, K, V = L_base.shape
    head = DominoHead({**weights, "W2": W2}, K=K, max_batch=B)

    def logits(tokens: torch.Tensor) -> torch.Tensor:
        out = head.draft(H, L_base, last_tok, teacher=tokens, want_logits=True)
        return torch.cat([out["L_final"], L_base[:, -1:]], 1)

    return logits


def main(workload: Optional[str] = None, steps: int = 8, beams: int = 4) -> dict:
    import domino_synth as ds

    from .tensors import device_tensor, head_weights_to_device

    w, inp = ds.make_workload(workload or "tiny")
    weights = head_weights_to_device(w)
    H, L_base, last_tok = (device_tensor(x) for x in (inp.H, inp.L_base, inp.last_tok))
    B, K, V = L_base.shape
    g = torch.Generator(device="cuda").manual_seed(1)
    spread = float(weights["W2"].float().std())
    noise = torch.randn(weights["W2"].shape, generator=g, device="cuda")
    other = (weights["W2"].float() + 2 * spread * noise).to(weights["W2"].dtype)
    target = synthetic_target(weights, other, H, L_base, last_tok)
    W2 = torch.nn.Parameter(weights["W2"].float().clone())
    optimizer, losses = torch.optim.AdamW([W2], lr=0.2 * spread), []
    for step in range(steps):
        got = distill_step(weights, W2, H, L_base, last_tok, target, k=min(64, V))
        optimizer.step()
        losses.append(float(got["loss"]))
        print("step %d: loss %.4f, mean accept length %.2f of %d" % (step, losses[-1], float(got["accept"]), K))
    one = DominoHead({**weights, "W2": W2.detach().to(weights["W2"].dtype)}, K=1, max_batch=B * beams)
    best = beam_draft(one, H, L_base, last_tok, beams)
    greedy = beam_draft(one, H, L_base, last_tok, 1)
    print("log-probability of the best of %d beams' drafts %.3f, of the greedy ones %.3f (means over %d rows)" %
          (beams, float(best["scores"][:, 0].mean()), float(greedy["scores"][:, 0].mean()), B))
    return {"losses": losses, "best": best, "greedy": greedy}


if __name__ == "__main__":
    main(*sys.argv[1:2])
