"""Distil the output head of a language model from a frozen teacher whose head
is held in 8 bits, with synthetic hidden states.

Each step:

  teacher   linear_i8        hidden states x 8-bit head -> logits
            token_logprobs   -> its top tokens and their log-probabilities
  student   Plan.gemm        hidden states x head -> logits
            distill_topk_grad  loss, and the gradient in place of the logits
            Plan.gemm        gradients of the head and of the hidden states
  checks    token_logprobs   the student's log-probability of the teacher's
                             first choice, and its entropy

Run:  python examples/distill_head.py [--steps 20 --tokens 512 --vocab 50001 --width 1024]
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import tensor_core_dense_tma_gb300 as tc  # noqa: E402


def run(steps: int = 20, tokens: int = 512, vocab: int = 50001, width: int = 1024, top: int = 32,
        temperature: float = 2.0, lr: float = 16.0, batches: int = 2,
        seed: int = 0, report=print) -> list[dict]:
    """The mean loss, agreement and entropy of each step, over `batches`
    batches of hidden states taken in turn."""
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    rows = -(-vocab // 8) * 8      # row stride of the logits: whole 16-byte units, as the products' loads want

    # the teacher: a head in 8 bits with a scale per vocabulary entry
    teacher = torch.randn((vocab, width), generator=g, device=dev) * (4.0 / width ** 0.5)
    teacher_q, teacher_scale = tc.quantize_rows_i8(teacher)
    # the student's head (fp32, its bf16 copy is multiplied), and the rows' weights: a mean over the tokens
    master = torch.zeros((vocab, width), device=dev)
    weight = torch.full((tokens,), 1.0 / tokens, device=dev)
    logits = torch.zeros((tokens, rows), dtype=torch.bfloat16, device=dev)[:, :vocab]
    teacher_logits = torch.empty((tokens, vocab), dtype=torch.bfloat16, device=dev)
    corpus = [torch.randn((tokens, width), generator=g, device=dev).bfloat16() for _ in range(batches)]
    history = []
    with tc.Plan("f16") as f16, tc.Plan("bf16") as bf16:
        for step in range(steps):
            h = corpus[step % batches]
            f16.linear_i8(h, teacher_q.t(), teacher_logits, col_scale=teacher_scale)
            best = tc.token_logprobs(teacher_logits, top=top)

            head = master.bfloat16()
            bf16.gemm(h, head.t(), None, logits)
            seen = tc.token_logprobs(logits, best.top_token[:, 0].contiguous())
            loss, dlogits = tc.distill_topk_grad(logits, best.top_token, best.top_logprob, weight,
                                                 temperature=temperature, dlogits=logits)
            d_head = bf16.gemm(dlogits.t(), h)              # vocab x width, fp32
            d_hidden = bf16.gemm(dlogits, head)             # what goes back into the student's body
            master -= (lr * tokens / width) * d_head        # |h|^2 is about the width
            history.append({"step": step, "loss": loss.mean().item(), "first_choice": seen.logprob.mean().item(),
                            "entropy": seen.entropy.mean().item(), "d_hidden": d_hidden.norm().item()})
            report("step {step:3d}  loss {loss:8.4f}  log p(teacher's first) {first_choice:8.4f}  "
                   "entropy {entropy:7.4f}  |d hidden| {d_hidden:.4g}".format(**history[-1]))
        torch.cuda.synchronize()
        assert f16.device_status() == 0 and bf16.device_status() == 0
    return history


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--vocab", type=int, default=50001)
    ap.add_argument("--width", type=int, default=1024)
    a = ap.parse_args()
    run(a.steps, a.tokens, a.vocab, a.width)


if __name__ == "__main__":
    main()
