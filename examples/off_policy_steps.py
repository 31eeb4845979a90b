"""More than one step on a batch of completions, then a preference step, on one lm_head (GB300).

    python examples/off_policy_steps.py [--d 1536 --V 151936 --L 256 --steps 3]

What a training loop around the library does with its log-prob and off-policy operators, on synthetic hidden states:

  1. record the sampling policy's and the frozen reference's log-probs of a group's completions (grpo_logprobs)
  2. several optimiser steps on that batch with the clipped policy loss (grpo_clip_loss_fwd_bwd)
  3. preference steps on pairs of completions, the better against the worse (grpo_pair_loss_fwd_bwd)
  4. the log-prob of one next token per completion, as while serving (grpo_logprobs, one row each)

The hidden states stand for a model's output and are stepped along their gradient; a real loop hands dH to the model.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import rl_fine_tuning_gb300 as rg  # noqa: E402


class Head:
    """Hidden states, lm_head weight and the buffers that the operators use, kept between calls."""

    def __init__(self, n_groups, G, L, d, V, beta=0.04, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        n = n_groups * G
        rnd = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
        self.shape = rg.make_shape(n_groups, G, L, d, V, beta=beta)
        self.W = (rnd(V, d) * d ** -0.5).bfloat16()
        self.tokens = torch.randint(0, V, (n * L,), device="cuda", generator=g, dtype=torch.int32)
        self.h_ref = (rnd(n * L, d) + 8 * self.W[self.tokens.long()].float()).bfloat16()
        self.h = (self.h_ref.float() + 0.05 * rnd(n * L, d)).bfloat16()
        self.lengths = torch.randint(max(1, L // 2), L + 1, (n,), device="cuda", generator=g, dtype=torch.int32)
        self.mask = torch.empty(n * L, dtype=torch.uint8, device="cuda")
        rg.grpo_build_mask(self.lengths, self.shape, self.mask)
        self.rewards = rnd(n)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.inf = torch.zeros_like(self.status)
        self.dH, self.dW = torch.empty_like(self.h), torch.empty_like(self.W)
        self.loss = torch.empty(1, device="cuda")
        self.ws = None

    def workspace(self, op):
        n = rg.grpo_policy_workspace_bytes(self.shape, op)
        if self.ws is None or self.ws.numel() < n:
            self.ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        return self.ws

    def logprobs(self, h):
        q, ent = torch.empty(2, self.shape.N, device="cuda").unbind(0)
        rg.grpo_logprobs(h, self.W, self.tokens, self.mask, self.shape, 1.0, self.workspace("logp"), q, ent, self.status)
        return q, ent

    def descend(self, lr):
        self.h.sub_((lr * self.dH.float()).to(self.h.dtype))
        self.W.sub_((lr * self.dW.float()).to(self.W.dtype))

    def check(self):
        if int(self.status) or int(self.inf):
            raise RuntimeError(f"{rg.grpo_status_string(int(self.status))}, found_inf {int(self.inf)}")


def clipped_steps(head, steps, lr):
    s = head.shape
    adv = torch.empty(s.n_groups * s.G, device="cuda")
    rg.grpo_group_advantages(head.rewards, s.n_groups, s.G, s.eps, bool(s.std_unbiased), adv)
    old, entropy = head.logprobs(head.h)
    ref, _ = head.logprobs(head.h_ref)
    stats = torch.empty(s.N, 3, device="cuda")
    opts = rg.clip_opts(clip_low=0.2, clip_high=0.28)
    losses = []
    for _ in range(steps):
        rg.grpo_clip_loss_fwd_bwd(head.h, head.W, head.tokens, head.mask, adv, old, ref, s, opts, 1.0, head.workspace("clip"),
                                  head.loss, head.dH, head.dW, head.inf, stats, head.status)
        head.check()
        losses.append(float(head.loss))
        head.descend(lr)
    on = head.mask.bool()
    ratio = stats[on, 1]
    return {"losses": losses, "entropy": float(entropy[on].mean()), "kl": float(stats[on, 2].mean()),
            "clipped": float(((ratio < 0.8) | (ratio > 1.28)).float().mean())}


def preference_steps(head, steps, lr):
    s = head.shape
    ref, _ = head.logprobs(head.h_ref)
    stats, logp = torch.empty(s.n_groups, 4, device="cuda"), torch.empty(s.N, device="cuda")
    losses = []
    for _ in range(steps):
        rg.grpo_pair_loss_fwd_bwd(head.h, head.W, head.tokens, head.mask, ref, s, rg.pair_opts(), 1.0, head.workspace("pair"),
                                  head.loss, head.dH, head.dW, head.inf, logp, stats, head.status)
        head.check()
        losses.append(float(head.loss))
        head.descend(lr)
    return {"losses": losses, "margin": float(stats[:, 2].mean())}


def serve_one_token(head, rows):
    """log-prob of one token for each of a few sequences: rows of the hidden states, no mask"""
    s = rg.make_shape(1, len(rows), 1, head.shape.d, head.shape.V)
    h, tok = head.h[rows].contiguous(), head.tokens[rows].contiguous()
    q = torch.empty(len(rows), device="cuda")
    ws = torch.empty(rg.grpo_policy_workspace_bytes(s, "logp"), dtype=torch.uint8, device="cuda")
    rg.grpo_logprobs(h, head.W, tok, None, s, 1.0, ws, q, None, head.status)
    head.check()
    return q


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, default in (("d", 1536), ("V", 151936), ("L", 256), ("steps", 3)):
        ap.add_argument("--" + name, type=int, default=default)
    a = ap.parse_args(argv)
    group = Head(1, 8, a.L, a.d, a.V)
    out = {"clip": clipped_steps(group, a.steps, lr=0.05)}
    pairs = Head(4, 2, a.L, a.d, a.V, beta=0.1, seed=1)
    out["pair"] = preference_steps(pairs, a.steps, lr=0.002)
    out["token"] = serve_one_token(group, [0, 1, 2]).tolist()
    for k, v in out.items():
        print(k, v)
    return out


if __name__ == "__main__":
    main()
