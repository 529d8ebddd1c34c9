"""The block operators on tensors whose offsets pass 32 bits: what the far rows,
columns and groups hold is that of the same call on them alone, bit for bit
(codes 0, 1 and -1 and scales 1 and 2, whose sums are exact, or values of which
each row is made alone)."""
import pytest
import torch

import bit_exact_fp8_amd as fw
from test_block_operators import E8, dev, exact_codes  # noqa: F401
from test_operators import BF, E4, SF, note, rand, rng


def bits(t):
    return t.contiguous().view(torch.uint8 if t.element_size() == 1 else torch.int16 if t.element_size() == 2 else torch.int32)


def alike(a, b):
    return torch.equal(bits(a), bits(b))


def strided(rows, ld, values):
    """values [rows, n] on the device as rows ld elements apart."""
    base = torch.empty((rows - 1) * ld + values.shape[1], dtype=torch.uint8 if values.dtype == E4 else values.dtype, device="cuda")
    v = base.as_strided((rows, values.shape[1]), (ld, 1))
    v.copy_(values.view(torch.uint8) if values.dtype == E4 else values)
    return v.view(values.dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [1, 128])
def test_block_quant_far(dev, rows):  # noqa: F811
    T, n = 33024, 65666
    note(f"block codes {T}x{n} rows={rows}")
    x = torch.zeros(T, n, dtype=BF, device=dev)
    x[-256:] = rand(rng(1), 256, n, dtype=BF).to(dev)
    q, s = fw.block_quant(x, block_rows=rows)
    assert q.numel() > 2 ** 31
    want_q, want_s = fw.block_quant(x[-256:].clone(), block_rows=rows)
    assert alike(q[-256:], want_q) and alike(s[-256 // rows:], want_s)
    assert not bits(q[-300:-256]).any()
    del q, s
    near = rand(rng(2), 3, 333, dtype=BF).to(dev)
    q, s = fw.block_quant(strided(3, 2 ** 30 + 7, near), block_rows=rows)
    want_q, want_s = fw.block_quant(near, block_rows=rows)
    assert alike(q, want_q) and alike(s, want_s)


@pytest.mark.gpu
def test_swiglu_far(dev):  # noqa: F811
    T, F = 33000, 32900
    note(f"gated activation {T}x{F}")
    both = torch.zeros(T, 2 * F, dtype=BF, device=dev)
    both[-5:] = rand(rng(1), 5, 2 * F, dtype=BF).to(dev)
    r = fw.swiglu_block_quant(both[:, :F], both[:, F:], keep=True)
    assert r.kept.numel() > 2 ** 31
    want = fw.swiglu_block_quant(both[-5:, :F].clone(), both[-5:, F:].clone(), keep=True)
    assert all(alike(a[-5:], b) for a, b in zip(r, want))
    d = fw.swiglu_block_backward(both[:, :F], r.kept, r.kept_scale)
    assert alike(d[-5:], fw.swiglu_block_backward(both[-5:, :F].clone(), want.kept, want.kept_scale)) and not d[:-5].any()


@pytest.mark.gpu
@pytest.mark.parametrize("out", [BF, SF])
def test_block_mm_far_outputs(dev, out):  # noqa: F811
    M, N, K = 33000, 65700, 128
    note(f"block product {M}x{N}x{K} {out}")
    (a, sa, av), (w, sw, wv) = exact_codes(rng(3), M, K, 1, E4, E8), exact_codes(rng(4), N, K, 128, E4, E8)
    y = fw.block_scaled_mm(a.to(dev), w.to(dev).t(), sa.to(dev), sw.to(dev).t(), out_dtype=out)
    assert y.numel() > 2 ** 31
    for rows in (slice(0, 70), slice(M - 70, M)):
        assert torch.equal(y[rows], (av[rows].to(dev) @ wv.t().contiguous().to(dev)).float().to(out))


@pytest.mark.gpu
def test_block_mm_far_operands(dev):  # noqa: F811
    """Rows 2^22 codes apart (the most that tiles take as they are) and more."""
    M, N, K = 1030, 300, 400
    for ld in (2 ** 22, 2 ** 22 + 16):
        note(f"block product {M}x{N}x{K}, rows {ld} apart")
        (a, sa, av), (w, sw, wv) = exact_codes(rng(5), M, K, 1, E4, E8), exact_codes(rng(6), N, K, 128, E4, E8)
        want = (av @ wv.t()).float().to(BF).to(dev)
        sa, sw = sa.to(dev), sw.to(dev)
        assert torch.equal(fw.block_scaled_mm(strided(M, ld, a.to(dev)), w.to(dev).t(), sa, sw.t()), want)
        # (and as the weights: the product turned over)
        (b, sb, bv), (v, sv, vv) = exact_codes(rng(7), N, K, 1, E4, E8), exact_codes(rng(8), M, K, 128, E4, E8)
        y = fw.block_scaled_mm(b.to(dev), strided(M, ld, v.to(dev)).t(), sb.to(dev), sv.to(dev).t())
        assert torch.equal(y, (bv @ vv.t()).float().to(BF).to(dev))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [40, 3000])
def test_grouped_far_weights(dev, T):  # noqa: F811
    E, N, K = 130, 4096, 4112
    note(f"grouped product {T}x{E}x{N}x{K}")
    (a, sa, av), (w, sw, wv) = exact_codes(rng(9), T, K, 1, E4, E8), exact_codes(rng(10), N, K, 128, E4, E8)
    codes = torch.zeros(E, N, K, dtype=torch.uint8, device=dev)
    codes[-1] = w.to(dev).view(torch.uint8)
    assert codes.numel() > 2 ** 31
    scales = sw.to(dev).view(torch.uint8).expand(E, -1, -1).contiguous().view(E8)
    first = T // 3
    ends = torch.full((E,), first, device=dev)
    ends[-1] = T
    y = fw.grouped_block_scaled_mm(a.to(dev), codes.view(E4).transpose(1, 2), sa.to(dev), scales.transpose(1, 2), ends)
    want = (av.to(dev) @ wv.t().contiguous().to(dev)).float().to(BF)
    assert torch.equal(y[first:], want[first:]) and not y[:first].any()


@pytest.mark.gpu
def test_weight_grad_far(dev):  # noqa: F811
    T, N, K = 70000, 32776, 130
    note(f"weights' gradient {T}x{N}x{K}")
    c, s, v = exact_codes(rng(11), T, K, 1, E4, E8)
    g = torch.zeros(T, N, dtype=BF, device=dev)
    g[-100:] = torch.randint(-2, 3, (100, N), generator=rng(12)).to(BF).to(dev)
    assert g.numel() > 2 ** 31
    y = fw.block_weight_grad(g, c.to(dev), s.to(dev), out_dtype=SF)
    want = g[-100:].double().t().contiguous() @ v[-100:].to(dev)
    assert torch.equal(y, want.float())
    del g, y
    E, T, N, K = 130, 2000, 4096, 4112
    note(f"weights' gradient {T}x{E}x{N}x{K}")
    c, s, v = exact_codes(rng(13), T, K, 1, E4, E8)
    g = torch.randint(-2, 3, (T, N), generator=rng(14)).to(BF).to(dev)
    ends = torch.full((E,), 1700, device=dev)
    ends[-1] = T
    y = fw.block_weight_grad(g, c.to(dev), s.to(dev), ends)
    assert y.numel() > 2 ** 31
    for e, rows in ((0, slice(0, 1700)), (E - 1, slice(1700, T))):
        assert torch.equal(y[e], (g[rows].double().t().contiguous() @ v[rows].to(dev)).float().to(BF))
    assert not y[1:-1].any()
