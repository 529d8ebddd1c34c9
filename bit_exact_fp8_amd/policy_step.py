"""The operators and the FP8 product together, as a training loop would run
them: a policy's last norm is fitted under a frozen 8-bit head.

    python -m bit_exact_fp8_amd.policy_step [--head int8|fp8] [--steps N]

A step adds a branch's output to the residual stream, normalises it into 8-bit
codes, multiplies them with the head's codes, takes the log probabilities of
the sampled tokens with the entropy and the most likely alternatives, and goes
back from the policy's loss to the gradients of the stream and of the norm's
weight.  The int8 head has a scale for each vocabulary entry and the codes one
for each token; the fp8 head goes through ``scaled_mm`` with one scale each,
the codes' left by calibration."""
from __future__ import annotations

import argparse
from typing import NamedTuple

import torch

from . import api, operators


class Head(NamedTuple):
    """A frozen vocabulary projection in 8 bits, codes [V, n]."""
    codes: torch.Tensor
    scale: torch.Tensor        # [1, V] (int8) or one value (fp8)
    in_scale: torch.Tensor | None  # fp8: the codes' scale that calibration left

    def weight(self) -> torch.Tensor:
        """What the codes stand for, float32 [V, n]."""
        return self.codes.float() * self.scale.reshape(-1, 1)


def int8_head(weight: torch.Tensor) -> Head:
    """Symmetric codes with a scale for each row of ``weight`` [V, n]."""
    scale = (weight.float().abs().amax(1, keepdim=True) / 127).clamp_min(2.0 ** -126)
    return Head((weight.float() / scale).round().to(torch.int8), scale.reshape(1, -1).contiguous(), None)


def fp8_head(weight: torch.Tensor, in_scale: float) -> Head:
    """e4m3fn codes with one scale, for normalised inputs with the scale ``in_scale``."""
    scale = (weight.float().abs().amax() / 448).clamp_min(2.0 ** -126).reshape(1)
    return Head((weight.float() / scale).to(torch.float8_e4m3fn), scale, torch.full_like(scale, in_scale))


class Step(NamedTuple):
    """What ``policy_step`` returns."""
    loss: torch.Tensor
    tokens: operators.TokenLogprobs
    grad_stream: torch.Tensor     # of the branch's output and of the residual alike
    grad_weight: torch.Tensor


@torch.no_grad()
def policy_step(branch: torch.Tensor, stream: torch.Tensor, norm_weight: torch.Tensor, head: Head, tokens: torch.Tensor,
                advantage: torch.Tensor, entropy_bonus: float = 0.01, top_k: int = 0,
                grad_stream: torch.Tensor | None = None) -> Step:
    """loss = mean(-advantage * logprob(token) - entropy_bonus * entropy) over the
    tokens [T], and its gradients; ``grad_stream``: what reaches the stream
    from elsewhere.  branch and stream [T, n], advantage float32 [T]."""
    T = branch.shape[0]
    out = torch.int8 if head.in_scale is None else torch.float8_e4m3fn
    codes, scale, h = operators.add_rms_norm_quant(branch, norm_weight, stream, out_dtype=out, scale=head.in_scale)
    if head.in_scale is None:
        logits = operators.int8_scaled_mm(codes, head.codes.t(), scale, head.scale, out_dtype=torch.float32)
    else:
        logits = api.scaled_mm(codes, head.codes.t(), scale, head.scale, out_dtype=torch.float32, use_fast_accum=True)
    r = operators.token_logprobs(logits, tokens, top_k=top_k)
    loss = -(advantage * r.logprobs + entropy_bonus * r.entropy).mean()
    grad_logits = operators.token_logprobs_backward(logits, tokens, r.lse, r.entropy, advantage / -T,
                                                    torch.full_like(r.entropy, -entropy_bonus / T), out=logits)
    # the rounding to 8 bits is passed straight through: dy = dz W
    grad_y = (grad_logits @ head.weight()).to(h.dtype)
    if h.dtype != branch.dtype:
        norm_weight = norm_weight.to(h.dtype)
    grad, grad_weight = operators.add_rms_norm_backward(grad_y, h, norm_weight, grad_h=grad_stream)
    return Step(loss, r, grad, grad_weight)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--head", choices=("int8", "fp8"), default="int8")
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--tokens", type=int, default=64)
    a = ap.parse_args(argv)
    V, n, T = 5760, 1920, a.tokens
    gen = torch.Generator(device="cuda").manual_seed(0)

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=gen, device="cuda") * std

    weight = normal(V, n, std=n ** -0.5)
    head = int8_head(weight) if a.head == "int8" else fp8_head(weight, 1 / 32)
    branch, stream = normal(T, n).bfloat16(), normal(T, n)
    norm_weight = torch.ones(n, device="cuda")
    tokens = torch.randint(0, V, (T,), generator=gen, device="cuda")
    advantage = torch.ones(T, device="cuda")
    for i in range(a.steps):
        s = policy_step(branch, stream, norm_weight, head, tokens, advantage, top_k=1)
        norm_weight -= 30.0 * s.grad_weight
        stream -= 30.0 * s.grad_stream
        hit = (s.tokens.top_tokens[:, 0] == tokens).float().mean()
        print(f"step {i}: loss {s.loss.item():.4f} entropy {s.tokens.entropy.mean().item():.4f} "
              f"most likely {hit.item():.2f}", flush=True)
    return s.loss.item()


if __name__ == "__main__":
    main()
