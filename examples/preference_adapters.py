"""Tune a low-rank adapter of a frozen output head on preferences, one on
rewards, and serve both and the head without an adapter in one batch; with
synthetic hidden states and preferences.

Each step:

  reference   linear_adapters       hidden states x head, no adapter -> logits
              token_logprobs        -> the reference's log-probabilities
  policy      linear_adapters       the same rows with their adapters -> logits
              preference_loss_grad  pairs of answers (adapter 0), gradient in place of the logits
              policy_loss_grad      sampled answers with advantages (adapter 1), likewise
              linear_adapters_grad  gradients of the factors and of the hidden states
serving       linear_adapters       single tokens of many requests, each with its adapter

Run:  python examples/preference_adapters.py [--steps 20 --tokens 256 --vocab 5003 --width 512]
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import tensor_core_dense_tma_gb300 as tc  # noqa: E402


def run(steps: int = 20, tokens: int = 256, vocab: int = 5003, width: int = 512, rank: int = 8, lr: float = 0.02,
        beta: float = 0.2, seed: int = 0, report=print, check=None) -> list[dict]:
    """Loss, margin and KL of each step.  tokens rows of preferences (pairs of answers of
    a sixteenth each) and as many of samples."""
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    rows = -(-vocab // 8) * 8      # row stride of the logits: whole 16-byte units, as the products' loads want
    pairs = max(1, tokens // 32)

    def normal(*shape, size):
        return (torch.randn(shape, generator=g, device=dev) * size)

    head = normal(vocab, width, size=width ** -0.5).bfloat16()
    hidden_states = normal(2 * tokens, width, size=1.0).bfloat16()
    answers = torch.randint(0, vocab, (2 * tokens,), generator=g, device=dev)
    # both adapters as they begin: up = 0, so the first step's policy is the reference
    down, up = normal(2, rank, width, size=width ** -0.5), torch.zeros((2, vocab, rank), device=dev)
    scale = torch.full((2,), 2.0, device=dev)
    none = torch.full((2 * tokens,), -1, dtype=torch.int32, device=dev)
    index = torch.arange(2 * tokens, device=dev).div(tokens, rounding_mode="floor").int()
    offsets = torch.linspace(0, tokens, 2 * pairs + 1, device=dev).long()
    advantage = torch.randn((tokens,), generator=g, device=dev)
    w_pair, w_token = torch.full((pairs,), 1 / pairs, device=dev), torch.full((tokens,), 1 / tokens, device=dev)
    logits = torch.zeros((2 * tokens, rows), dtype=torch.bfloat16, device=dev)[:, :vocab]
    m = [torch.zeros_like(down), torch.zeros_like(up)]
    history = []
    with tc.Plan("bf16") as plan:
        lower, upper = down.bfloat16(), up.bfloat16()
        plan.linear_adapters(hidden_states, head.t(), lower, upper, none, scale, logits)
        ref = tc.token_logprobs(logits, answers).logprob
        for step in range(steps):
            lower, upper = down.bfloat16(), up.bfloat16()
            _, kept = plan.linear_adapters(hidden_states, head.t(), lower, upper, index, scale, logits)
            seen = logits.clone() if check else None
            pref = tc.preference_loss_grad(logits[:tokens], answers[:tokens], offsets, w_pair, ref[:tokens], beta=beta,
                                           dlogits=logits[:tokens])
            pol = tc.policy_loss_grad(logits[tokens:], answers[tokens:], ref[tokens:], advantage, w_token, ref[tokens:],
                                      clip=(0.2, 0.28), kl=0.05, entropy_bonus=0.001, dlogits=logits[tokens:])
            grads = plan.linear_adapters_grad(logits, head.t(), hidden_states, kept, lower, upper, index, scale,
                                              d_down=torch.empty_like(down), d_up=torch.empty_like(up))
            if check:
                check(dict(seen=seen, dlogits=logits, answers=answers, offsets=offsets, ref=ref, advantage=advantage,
                           beta=beta, head=head, hidden_states=hidden_states, lower=lower, upper=upper, index=index,
                           scale=scale, w_pair=w_pair, w_token=w_token, grads=grads, pref=pref, pol=pol))
            for p, d, v in zip((down, up), (grads.d_down, grads.d_up), m):
                v.mul_(0.9).add_(d / d.square().mean().sqrt().clamp(min=1e-12), alpha=0.1)
                p -= lr * rank ** -0.5 * 0.1 * v
            history.append({"step": step, "preference": pref.loss.mean().item(), "policy": pol.loss.mean().item(),
                            "margin": (pref.reward[0::2] - pref.reward[1::2]).mean().item(), "kl": pol.kl.mean().item(),
                            "d_hidden": grads.dX.float().norm().item()})
            report("step {step:3d}  preference {preference:8.4f}  margin {margin:8.4f}  policy {policy:8.4f}  "
                   "KL {kl:8.5f}  |d hidden| {d_hidden:.4g}".format(**history[-1]))
        # one token of each of many requests: adapter 0, 1 or none
        lower, upper = down.bfloat16(), up.bfloat16()
        which = (torch.arange(24, device=dev) % 3 - 1).int()
        served, _ = plan.linear_adapters(hidden_states[:24], head.t(), lower, upper, which, scale, out_dtype="f32")
        history.append({"served": served, "which": which, "state": (hidden_states[:24], head, lower, upper, scale)})
        torch.cuda.synchronize()
        assert plan.device_status() == 0
    return history


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--tokens", type=int, default=256)
    ap.add_argument("--vocab", type=int, default=5003)
    ap.add_argument("--width", type=int, default=512)
    a = ap.parse_args()
    run(a.steps, a.tokens, a.vocab, a.width)


if __name__ == "__main__":
    main()
