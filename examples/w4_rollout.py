"""A rollout and a training step with a 4-bit LM head (synthetic weights and states).

Rollout: the head is quantised to 4 bits once per policy; every decode step is one call,
logprob_w4, which gives each sequence's token its log probability, the entropy of the
distribution it came from and the most likely alternatives, here under a mask of allowed
tokens.  Training: the same rows in one batch (their bits do not depend on the batch, so
the two sides' log probabilities agree exactly), a policy loss with an entropy bonus, and
its gradient with respect to the logits and the hidden states.

    python examples/w4_rollout.py [--sequences 8] [--steps 16] [--hidden 4096] [--vocab 151936]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import invariant_token_logprob_gb300 as rlk  # noqa: E402
from invariant_token_logprob_gb300.inputs import lm_head_inputs  # noqa: E402


def allowed_bits(keep):
    """bool [T, V] -> the packed words of allowed-token bits."""
    T, V = keep.shape
    words = (V + 31) // 32
    padded = torch.zeros(T, words * 32, dtype=torch.bool, device=keep.device)
    padded[:, :V] = keep
    bits = torch.zeros(T, words, dtype=torch.int32, device=keep.device)
    for b in range(32):
        bits |= padded[:, b::32].to(torch.int32) << b
    return bits


def run(sequences=8, steps=16, hidden=4096, vocab=151936, top_k=20, group=128, seed=0):
    T = sequences * steps
    d = lm_head_inputs(T, hidden, vocab, seed=seed, device="cuda")
    h = d["h"]  # row s * sequences + i: the state of sequence i at step s
    codes, scales, zeros = rlk.quantize_w4(d["W"], group=group, asymmetric=True)

    # ---- rollout: the most likely allowed token, chosen from the alternatives
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    keep = torch.rand(T, vocab, generator=g, device="cuda") < 0.9
    allowed = allowed_bits(keep)
    logits = torch.empty(sequences, vocab, device="cuda")
    tokens = torch.empty(T, dtype=torch.int32, device="cuda")
    rollout = torch.empty(T, device="cuda")
    for s in range(steps):
        rows = slice(s * sequences, (s + 1) * sequences)
        step = rlk.logprob_w4(h[rows], codes, scales, d["targets"][rows], zeros=zeros, group=group,
                              top_k=top_k, allowed=allowed[rows], logits=logits)
        tokens[rows], rollout[rows] = step.top_ids[:, 0], step.top_logp[:, 0]

    # ---- training: all rows at once, gradient of a policy loss with an entropy bonus
    z = rlk.linear_w4(h, codes, scales, zeros, group).requires_grad_()
    out = rlk.differentiable_token_logprobs(z, tokens, 0, allowed)
    stats = rlk.consistency_stats(out.logp.detach(), rollout)
    advantage = torch.randn(T, generator=g, device="cuda")
    loss = -(advantage * out.logp).mean() - 0.01 * out.entropy.mean()
    loss.backward()
    W = rlk.dequantize_w4(codes, scales, zeros, group)
    grad_h = z.grad.to(torch.bfloat16) @ W  # the frozen head's input gradient
    rlk.check_device_error()
    return dict(loss=float(loss.detach()), stats=stats, entropy=float(out.entropy.detach().mean()), grad_z=z.grad,
                grad_h=grad_h, tokens=tokens, keep=keep)


def main():
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--sequences", type=int, default=8)
    p.add_argument("--steps", type=int, default=16)
    p.add_argument("--hidden", type=int, default=4096)
    p.add_argument("--vocab", type=int, default=151936)
    a = p.parse_args()
    r = run(a.sequences, a.steps, a.hidden, a.vocab)
    print(f"loss {r['loss']:.4f}, mean entropy {r['entropy']:.3f}, |grad h| {float(r['grad_h'].norm()):.3g}")
    print("rollout against training:", r["stats"])


if __name__ == "__main__":
    main()
