"""The block operators under the least and the largest scales of either type,
against their definitions in 64 bits."""
import math

import pytest
import torch

import bit_exact_fp8_amd as fw
from test_block_operators import E8, blocks, dev, exact_codes, kept_values, spread, swiglu_grad64  # noqa: F401
from test_operators import BF, E4, E5, F, HF, INF, SF, close, f64, half_step, note, rand, rng, wide

# (of a's blocks, of w's): products of a scale pair and of whole values stay within binary32
PAIRS = [(0, 127), (127, 0), (0, 254), (254, 0), (1, 120), (64, 70), (240, 120), (180, 180)]


def value(byte):
    return math.nan if byte == 255 else 2.0 ** (byte - 127)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K,pad", [(3, 70, 300, 0), (3, 70, 300, 3), (40, 130, 256, 3), (200, 300, 384, 0), (1100, 1200, 256, 0),
                                       (2100, 2300, 128, 0)])
@pytest.mark.parametrize("out", [BF, SF])
@pytest.mark.parametrize("scale", [E8, SF])
def test_block_mm_of_far_scales(dev, M, N, K, pad, out, scale):  # noqa: F811
    """Codes 0, 1 and -1 under one pair of scales each: whole numbers times a
    power of two, which binary32 holds wherever it is normal."""
    gen = rng(M)
    a, _, _ = exact_codes(gen, M, K, 1, E4, E8)
    w, _, _ = exact_codes(gen, N, K, 128, E5, E8)
    sums = (a.to(f64) @ w.to(f64).t()).to(dev)
    a = wide(a.view(torch.uint8), pad, dev).view(E4)
    for i, j in PAIRS:
        note(f"block product {M}x{N}x{K} {out} {scale} under scales of {i} and {j}")
        sa = torch.full((M, blocks(K)), i, dtype=torch.uint8, device=dev).view(E8).to(SF).to(scale)
        sw = torch.full((blocks(N), blocks(K)), j, dtype=torch.uint8, device=dev).view(E8).to(SF).to(scale)
        y = fw.block_scaled_mm(a, w.to(dev).t(), sa, sw.t(), out_dtype=out)
        want = (sums * (value(i) * value(j))).to(SF).to(out)
        assert torch.equal(y, want), (i, j, (y != want).nonzero()[:3].tolist(), y[y != want][:3], want[y != want][:3])


@pytest.mark.gpu
@pytest.mark.parametrize("code", [E4, E5])
@pytest.mark.parametrize("T,N,K", [(64, 64, 256), (64, 300, 4200)])
def test_weight_grad_of_every_scale(dev, code, T, N, K):  # noqa: F811
    """Each row has a scale of its own, and each output comes from one row: what
    bf16 holds of code times scale, from 2^-133 on and below infinity."""
    for low in range(0, 255, T):
        bytes_ = torch.arange(low, low + T).clamp_max(254)
        note(f"weights' gradient under scales from {low} on, {code}")
        c = torch.tensor([1.0, -1.0, 1.5, 0.5, -1.75])[torch.randint(0, 5, (T, K), generator=rng(low))].to(code)
        s = bytes_.to(torch.uint8)[:, None].expand(T, blocks(K)).contiguous()
        g = torch.zeros(T, N)
        g.fill_diagonal_(1.0)
        y = fw.block_weight_grad(g.bfloat16().to(dev), c.to(dev), s.view(E8).to(dev), out_dtype=SF).cpu()
        x = c.to(f64) * torch.exp2((bytes_ - 127).to(f64))[:, None]
        # (subnormal numbers of bf16 end at 2^-133, those of these codes at 2^-129 and 1.75 of it)
        assert torch.equal(y[:T].to(f64), x.float().to(BF).to(f64)), low


@pytest.mark.gpu
@pytest.mark.parametrize("byte", [0, 1, 20, 250, 254])
def test_swiglu_grad_of_far_scales(dev, byte):  # noqa: F811
    """Up's values near either end of binary32: the gradient toward gate is theirs, in proportion."""
    n = 200
    a, _, _ = exact_codes(rng(byte), 5, n, 1, E4, E8)
    kept = torch.cat([torch.ones(5, n).to(E4).view(torch.uint8), a.view(torch.uint8)], 1).view(E4)
    s = torch.tensor([127, 127, byte, byte], dtype=torch.uint8).expand(5, 4).contiguous().view(E8)
    g = torch.full((5, n), 0.5)
    d = fw.swiglu_block_backward(g.to(dev), kept.to(dev), s.to(dev))
    gate, up = kept_values(kept, s, n)
    want = swiglu_grad64(g.to(f64), gate, up)
    close(d, want, half_step(want, SF) + F * want.abs() + 3 * 2.0 ** -149, "gradient")
