"""A training step of a layer of experts on 8-bit codes with a scale for each
block of 128, forward and back:

    python -m bit_exact_fp8_amd.expert_step [--experts E] [--steps N]

Rows are sorted by the expert that a router chose for them.  Forward: codes of
the rows, the product with each expert's gate and up projections, the gated
activation as codes, the product with its down projection.  What is kept for
the gradient is in 8 bits: the rows' codes, the activation's, and those of gate
and up.  Back: the weights' gradients from the kept codes, the inputs' from
codes of the gradients and the weights' codes laid out the other way."""
from __future__ import annotations

import argparse
from typing import NamedTuple

import torch

from . import block_operators as ops


class Projection(NamedTuple):
    """Experts' weights [E, N, K] in blocks of 128 x 128, and the same [E, K, N]."""
    codes: torch.Tensor
    scale: torch.Tensor
    turned: torch.Tensor
    turned_scale: torch.Tensor


def project(weight: torch.Tensor, out_dtype=torch.float8_e4m3fn) -> Projection:
    """Codes of ``weight`` [E, N, K]: a block keeps its scale when it is turned."""
    codes, scale = ops.block_quant(weight, block_rows=ops.BLOCK, out_dtype=out_dtype)
    return Projection(codes, scale, _turned(codes), _turned(scale))


def _turned(t: torch.Tensor) -> torch.Tensor:
    return t.view(torch.uint8).transpose(1, 2).contiguous().view(t.dtype)


def _product(codes, scale, weight, weight_scale, ends, out_dtype):
    return ops.grouped_block_scaled_mm(codes, weight.transpose(1, 2), scale, weight_scale.transpose(1, 2), ends,
                                       out_dtype=out_dtype)


def _joined(rows, order, T, c):
    """[T, n]: of rows by expert each token's c, added in the order of its choices."""
    at = torch.empty_like(order)
    at[order] = torch.arange(T * c, device=order.device)
    rows = rows[at].view(T, c, rows.shape[1])
    out = rows[:, 0] if c else rows.new_zeros(T, rows.shape[2])
    for j in range(1, c):
        out = out + rows[:, j]
    return out


class Kept(NamedTuple):
    """What the forward pass leaves for the gradient."""
    order: torch.Tensor        # the rows' places among (token, choice), by expert
    ends: torch.Tensor         # each expert's last row, and one
    x: torch.Tensor            # the rows' codes and scales
    x_scale: torch.Tensor
    h: ops.SwigluCodes


@torch.no_grad()
def forward(x: torch.Tensor, up: Projection, down: Projection, choice: torch.Tensor, share: torch.Tensor):
    """(output [T, n] of x's type, what the gradient needs): the sum over each
    token's choices of ``share * expert(x)``.

    x [T, n]; up: gate's and up's projections [E, 2 F, n], down [E, n, F];
    choice [T, c] the experts of each token, share [T, c] float32."""
    T, c = choice.shape
    flat = choice.reshape(-1)
    order = torch.argsort(flat, stable=True)
    E = up.codes.shape[0]
    ends = torch.bincount(flat, minlength=E).cumsum(0)
    codes, scale = ops.block_quant(x[order // c])
    both = _product(codes, scale, up.codes, up.scale, ends, x.dtype)
    F = both.shape[1] // 2
    h = ops.swiglu_block_quant(both[:, :F], both[:, F:], keep=True)
    y = _product(h.codes, h.scale, down.codes, down.scale, ends, torch.float32)
    out = _joined(y * share.reshape(-1)[order, None], order, T, c)
    return out.to(x.dtype), Kept(order, ends, codes, scale, h)


class Gradients(NamedTuple):
    x: torch.Tensor
    up: torch.Tensor      # float32, of the weights in full
    down: torch.Tensor


@torch.no_grad()
def backward(grad: torch.Tensor, kept: Kept, up: Projection, down: Projection, share: torch.Tensor) -> Gradients:
    """The gradients of ``forward``'s output with respect to x and both
    projections, roundings to 8 bits passed straight through; ``grad`` [T, n]."""
    T, c = share.shape
    rows = (grad.float()[kept.order // c] * share.reshape(-1)[kept.order, None]).to(grad.dtype)
    grad_down = ops.block_weight_grad(rows, kept.h.codes, kept.h.scale, kept.ends, out_dtype=torch.float32)
    codes, scale = ops.block_quant(rows)
    grad_h = _product(codes, scale, down.turned, down.turned_scale, kept.ends, grad.dtype)
    grad_both = ops.swiglu_block_backward(grad_h, kept.h.kept, kept.h.kept_scale)
    grad_up = ops.block_weight_grad(grad_both, kept.x, kept.x_scale, kept.ends, out_dtype=torch.float32)
    codes, scale = ops.block_quant(grad_both)
    grad_rows = _product(codes, scale, up.turned, up.turned_scale, kept.ends, torch.float32)
    return Gradients(_joined(grad_rows, kept.order, T, c).to(grad.dtype), grad_up, grad_down)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--experts", type=int, default=8)
    ap.add_argument("--steps", type=int, default=10)
    ap.add_argument("--tokens", type=int, default=512)
    a = ap.parse_args(argv)
    n, F, E, T = 1920, 1024, a.experts, a.tokens
    gen = torch.Generator(device="cuda").manual_seed(0)

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=gen, device="cuda") * std

    weight_up, weight_down = normal(E, 2 * F, n, std=n ** -0.5), normal(E, n, F, std=F ** -0.5)
    x, target = normal(T, n).bfloat16(), normal(T, n)
    likely, choice = normal(T, E).softmax(1).topk(min(2, E), 1)
    share = likely / likely.sum(1, keepdim=True)
    for i in range(a.steps):
        up, down = project(weight_up), project(weight_down)
        out, kept = forward(x, up, down, choice, share)
        off = out.float() - target
        loss = off.square().mean()
        # the gradient of half the sum over a token's values, in the mean over tokens
        g = backward((off / T).bfloat16(), kept, up, down, share)
        weight_up -= 0.2 * g.up
        weight_down -= 0.2 * g.down
        print(f"step {i}: loss {loss.item():.4f}", flush=True)
    return loss.item()


if __name__ == "__main__":
    main()
