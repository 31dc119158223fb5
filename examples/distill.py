"""Distillation from a teacher whose head runs in 8 bits, the student trained by Dion3.

    python examples/distill.py [--steps 30] [--bits 4]

One training step, on synthetic tokens:
  teacher (frozen)  residual + RMS norm written as 8-bit codes -> 8-bit product with the head -> its top logits
  student           a linear layer, residual + RMS norm, a 16-bit head -> the loss on the teacher's top logits
  backward          the loss' gradient and the norm's from the library, the products' from torch
  update            Dion3 for the matrices, plain SGD for the norm's weight
Some tokens (the first eighth, as a prompt's) have no teacher: their loss and gradients are zero.

With --bits 4 both are layer-norm models and the teacher's head runs in 4-bit floating point:
  teacher (frozen)  residual + layer norm -> 4-bit codes -> 4-bit product with the head -> its top log probabilities
  student           residual + layer norm, the loss on them, and a share of the loss of the teacher's first token with a
                    bonus on the entropy
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import orthogonalized_optimizer_step_amd as dion  # noqa: E402


def main(steps=30, tokens=1024, dim=256, vocab=3001, k=48, temperature=2.0, seed=0, lr_layer=0.05, lr_head=0.2, bits=8):
    """Trains for `steps` steps and returns the mean loss of each."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    randn = lambda *shape: torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)

    # the teacher: its weights are quantised once, a scale for each output channel
    layer_t = randn(dim, dim) / dim ** 0.5
    norm_t = 1 + 0.1 * randn(dim)
    quantize = dion.int8_quantize if bits == 8 else dion.mxfp4_quantize
    head_t, head_scale = quantize(randn(vocab, dim) * 0.3)
    shift_t = 0.1 * randn(dim) if bits == 4 else None

    # the student
    layer = torch.nn.Parameter(randn(dim, dim).mul_(0.2 / dim ** 0.5))
    head = torch.nn.Parameter(torch.zeros(vocab, dim, device="cuda", dtype=torch.bfloat16))
    norm = torch.nn.Parameter(torch.ones(dim, device="cuda", dtype=torch.bfloat16))
    shift = torch.nn.Parameter(torch.zeros(dim, device="cuda", dtype=torch.bfloat16))
    matrices = dion.Dion3([{"params": [layer], "lr": lr_layer}, {"params": [head], "lr": lr_head}], momentum=0.9,
                          row_frac=1.0)
    vectors = torch.optim.SGD([norm] if bits == 8 else [norm, shift], lr=0.1)

    losses = []
    for _ in range(steps):
        x = randn(tokens, dim)
        with torch.no_grad():
            if bits == 8:
                codes, scale, _ = dion.rmsnorm_int8(x @ layer_t.t(), norm_t, residual=x)
                logits_t = dion.int8_linear(codes, scale, head_t, head_scale, out_dtype=torch.float32)
                top, index = logits_t.topk(k)
            else:
                codes, scale = dion.mxfp4_quantize(dion.layernorm(x @ layer_t.t(), norm_t, shift_t, residual=x)[0])
                logits_t = dion.mxfp4_linear(codes, scale, head_t, head_scale, out_dtype=torch.float32)
                top, index = dion.top_logprobs(logits_t, k)[:2]
            index[: tokens // 8] = -1
        if bits == 8:
            y, _ = dion.rms_norm(x @ layer.t(), norm, x)
        else:
            y, _ = dion.layer_norm(x @ layer.t(), norm, shift, x)
        logits = y @ head.t()
        per_token = dion.distill_loss(logits, top, index, temperature)
        if bits == 4:
            logprob, entropy = dion.log_probs(logits, index[:, 0])
            per_token = per_token - 0.1 * logprob - 0.001 * entropy * (index[:, 0] >= 0)
        loss = per_token.sum() / (tokens - tokens // 8)
        matrices.zero_grad()
        vectors.zero_grad()
        loss.backward()
        matrices.step()
        vectors.step()
        losses.append(float(loss.detach()))
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=30)
    ap.add_argument("--bits", type=int, choices=(8, 4), default=8)
    args = ap.parse_args()
    for i, value in enumerate(main(args.steps, bits=args.bits)):
        print(f"step {i:3d}  loss {value:.4f}")
