"""The operators of include/emu_operators.h against their definitions in 64
bits: the norm with 8-bit codes and its gradient, the int8 product, token log
probabilities and their gradient; and their refusals (on the CPU).

Tolerances, from the arithmetic: a stored value is rounded once, by
finfo.eps / 2 of it.  Before that every kernel works in binary32, a value
passing through at most some 10 operations and a sum through at most 64
additions in a row (the rest is a tree), each off by 2^-24 of its size:
F = 80 * 2^-24 of the terms' absolute sum bounds it."""
import math

import pytest
import torch

import bit_exact_fp8_amd as fw
from bit_exact_fp8_amd import operators

F = 80 * 2.0 ** -24
f64 = torch.float64
BF, HF, SF = torch.bfloat16, torch.float16, torch.float32
E4, E5, I8 = torch.float8_e4m3fn, torch.float8_e5m2, torch.int8
MOST = {E4: 448.0, E5: 57344.0, I8: 127.0}
INF = math.inf


def note(msg):
    print("[gpu] " + msg, flush=True)


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def rng(seed):
    return torch.Generator().manual_seed(seed)


def rand(gen, *shape, std=1.0, dtype=SF):
    return (torch.randn(shape, generator=gen) * std).to(dtype)


def wide(t, pad, dev, fill=7.0):
    """`t` on the device as rows of a wider matrix: another row stride, and another alignment."""
    if pad == 0:
        return t.to(dev)
    big = torch.full((t.shape[0], t.shape[1] + pad), fill, dtype=SF).to(t.dtype)
    big[:, 1:1 + t.shape[1]] = t
    return big.to(dev)[:, 1:1 + t.shape[1]]


def close(got, want, tol, what):
    """|got - want| <= tol, elementwise; infinities and NaN in the same places."""
    got, want, tol = got.detach().cpu().to(f64), want.cpu().to(f64), tol.cpu().to(f64)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert torch.equal(got.isnan(), want.isnan()), what + ": NaN in other places"
    inf = want.isinf()
    assert torch.equal(got[inf], want[inf]), what + ": infinities"
    fine = want.isfinite()
    over = ((got - want).abs() - tol)[fine]
    assert not over.numel() or float(over.max()) <= 0, f"{what}: {float(over.max())} over the tolerance"


def half_step(t, dtype):
    """Half a step of `dtype` at the values t (normal and subnormal)."""
    fi = torch.finfo(dtype)
    return t.abs().to(f64) * (fi.eps / 2) + fi.smallest_normal * fi.eps / 2


# ---- the norm ---------------------------------------------------------------
def norm64(x, res, w, eps):
    v = x.to(f64) if res is None else x.to(f64) + res.to(f64)
    r = 1.0 / (v.pow(2).mean(1, keepdim=True) + eps).sqrt()
    return v, v * r * w.to(f64)


def check_norm(dev, T, n, x_t, r_t, out, given, pad=0, w_t=None, seed=0, inplace=False, eps=1e-6):
    g = rng(seed)
    x = rand(g, T, n, dtype=x_t)
    res = None if r_t is None else rand(g, T, n, std=2.0, dtype=r_t)
    w = (1 + rand(g, n, std=0.2)).to(w_t or x_t)
    scale = torch.tensor([2.5 / MOST[out]]) if given else None
    note(f"norm {T}x{n} {x_t} {r_t} {out} given={given} pad={pad}")
    xd, wd = wide(x, pad, dev), w.to(dev)
    rd = None if res is None else wide(res, pad, dev)
    q, s, h = fw.add_rms_norm_quant(xd, wd, rd, eps=eps, out_dtype=out, scale=None if scale is None else scale.to(dev),
                                    h_out=rd if inplace else None)
    torch.cuda.synchronize(dev)
    v, y = norm64(x, res, w, eps)
    assert q.dtype == out and q.shape == x.shape
    if res is None:
        assert h is None
    else:
        want = (x.float() + res.float()).to(r_t)
        assert h.dtype == r_t and torch.equal(h.cpu(), want)
        if inplace:
            assert h.data_ptr() == rd.data_ptr()
    if given:
        assert s.shape == (1,)
    else:
        assert s.shape == (T, 1) and s.dtype == SF
        want = (y.abs().amax(1, keepdim=True) / MOST[out]).clamp_min(2.0 ** -126) if T else torch.zeros(0, 1)
        close(s, want, want * F, "scale")
    if not T:
        return
    s64 = s.cpu().to(f64)
    z = (y / s64).clamp(-MOST[out], MOST[out])
    step = torch.full_like(z, 0.5) if out == I8 else half_step(z, out)
    close(q.cpu().float(), z, step + z.abs() * F, "codes")


NORM = [(1, 1), (1, 7), (5, 8), (3, 64), (4, 511), (9, 512), (5, 513), (7, 1024), (2, 1025), (33, 1925), (3, 2048),
        (2, 2049), (3, 4096), (2, 4097), (3, 8192), (2, 8193), (2, 16384), (2, 16385), (1, 40000), (0, 64)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,n", NORM)
@pytest.mark.parametrize("x_t,r_t,out,given", [(BF, BF, E4, True), (BF, SF, I8, False), (HF, HF, E5, False),
                                               (SF, SF, E4, False), (HF, None, I8, True), (HF, SF, E4, False),
                                               (BF, None, E5, True), (SF, None, I8, False)])
def test_norm(dev, T, n, x_t, r_t, out, given):
    check_norm(dev, T, n, x_t, r_t, out, given)


@pytest.mark.gpu
@pytest.mark.parametrize("pad", [2, 3, 8])
@pytest.mark.parametrize("n", [7, 520, 1920, 4100, 17000])
def test_norm_strides_and_in_place(dev, n, pad):
    check_norm(dev, 6, n, BF, BF, I8, False, pad=pad, seed=3)
    check_norm(dev, 6, n, HF, SF, E4, True, pad=pad, w_t=SF, seed=4, inplace=True)


@pytest.mark.gpu
def test_norm_leading_axes(dev):
    g = rng(5)
    x, w = rand(g, 2, 3, 96, dtype=BF).to(dev), rand(g, 96, dtype=BF).to(dev)
    q, s, h = fw.add_rms_norm_quant(x, w, x, out_dtype=I8)
    q2, s2, h2 = fw.add_rms_norm_quant(x.view(6, 96), w, x.view(6, 96), out_dtype=I8)
    assert q.shape == (2, 3, 96) and s.shape == (2, 3, 1) and h.shape == (2, 3, 96)
    assert torch.equal(q.view(6, 96), q2) and torch.equal(s.view(6, 1), s2) and torch.equal(h.view(6, 96), h2)


@pytest.mark.gpu
@pytest.mark.parametrize("out", [E4, E5, I8])
@pytest.mark.parametrize("n", [40, 2000, 20000])
def test_norm_special_rows(dev, out, n):
    """Zeros, an infinity, a NaN and huge values: each row by itself."""
    x = rand(rng(6), 5, n)
    x[0] = 0
    x[1, n // 2] = INF
    x[2, n - 1] = math.nan
    x[3] *= 1e15
    w = torch.ones(n)
    for given in (None, torch.tensor([0.01], device=dev)):
        q, s, _ = fw.add_rms_norm_quant(x.to(dev), w.to(dev), out_dtype=out, scale=given)
        q = q.cpu().float()
        assert (q[0] == 0).all()
        v, y = norm64(x[3:], None, w, 1e-6)
        if given is None:
            s = s.cpu()
            assert s[0] == 2.0 ** -126 and s[1].isnan() and s[2].isnan()
            assert torch.equal(q[1:3].isnan(), torch.full((2, n), out != I8)) and (out != I8 or (q[1:3] == 0).all())
            sc = s[3:].to(f64)
        else:
            # 1 / sqrt(inf) is 0: finite values become 0, the infinity NaN
            assert (q[1, :n // 2] == 0).all() and (q[1, n // 2].isnan() or out == I8)
            assert torch.equal(q[2].isnan(), torch.full((n,), out != I8))
            sc = torch.full((2, 1), float(given.cpu()), dtype=f64)
        z = (y / sc).clamp(-MOST[out], MOST[out])
        step = torch.full_like(z, 0.5) if out == I8 else half_step(z, out)
        close(q[3:], z, step + z.abs() * F, "other rows")


@pytest.mark.gpu
def test_norm_feeds_the_fp8_product(dev):
    """One calibrated scale: codes and scale go into scaled_mm as they are."""
    g = rng(7)
    x, w = rand(g, 16, 256, dtype=BF).to(dev), torch.ones(256, dtype=BF, device=dev)
    sc = torch.tensor([4.0 / 448], device=dev)
    q, s, _ = fw.add_rms_norm_quant(x, w, scale=sc)
    w8 = rand(g, 64, 256).to(E4).to(dev)
    one = torch.ones(1, device=dev)
    y = fw.scaled_mm(q, w8.t(), s, one, out_dtype=SF, use_fast_accum=False)
    want = (q.cpu().double() @ w8.cpu().double().t()) * float(sc.cpu())
    # the emulated sums keep 13 fraction bits of each block's largest term
    assert float((y.cpu().double() - want).abs().max()) < 0.02 * float(want.abs().max())


# ---- the norm's gradient ----------------------------------------------------
def norm_grad64(g, h, w, eps, gh):
    g, h, w = g.to(f64), h.to(f64), w.to(f64)
    n = h.shape[1]
    r = 1.0 / (h.pow(2).mean(1, keepdim=True) + eps).sqrt()
    u, hn = g * w, h * r
    d = r * (u - hn * (u * hn).mean(1, keepdim=True))
    size = r * (u.abs() + hn.abs() * (u * hn).abs().mean(1, keepdim=True))
    if gh is not None:
        d, size = d + gh.to(f64), size + gh.to(f64).abs()
    return d, size, (g * hn).sum(0), (g * hn).abs().sum(0)


def check_norm_grad(dev, T, n, g_t, h_t, gh_t, w_t, pad=0, seed=0):
    gen = rng(seed)
    g, h = rand(gen, T, n, std=0.1, dtype=g_t), rand(gen, T, n, std=1.5, dtype=h_t)
    w = (1 + rand(gen, n, std=0.2)).to(w_t)
    gh = None if gh_t is None else rand(gen, T, n, std=0.1, dtype=gh_t)
    note(f"norm gradient {T}x{n} {g_t} {h_t} {gh_t} pad={pad}")
    gi, gw = fw.add_rms_norm_backward(wide(g, pad, dev), wide(h, pad, dev), w.to(dev),
                                      grad_h=None if gh is None else wide(gh, pad, dev))
    torch.cuda.synchronize(dev)
    d, size, dw, dw_size = norm_grad64(g, h, w, 1e-6, gh)
    assert gi.dtype == g_t and gw.dtype == w_t
    close(gi, d, half_step(d, g_t) + size * F, "grad_in")
    close(gw, dw, half_step(dw, w_t) + dw_size * F, "grad_weight")


@pytest.mark.gpu
@pytest.mark.parametrize("T,n", [(t, n) for t, n in NORM] + [(1500, 64), (700, 1100), (600, 5000)])
@pytest.mark.parametrize("g_t,h_t,gh_t,w_t", [(BF, BF, BF, BF), (BF, SF, SF, BF), (HF, HF, None, SF), (SF, SF, SF, SF),
                                              (HF, SF, HF, HF)])
def test_norm_grad(dev, T, n, g_t, h_t, gh_t, w_t):
    check_norm_grad(dev, T, n, g_t, h_t, gh_t, w_t)


@pytest.mark.gpu
@pytest.mark.parametrize("pad", [2, 3, 8])
@pytest.mark.parametrize("n", [9, 1000, 1925, 4100, 12000, 17000])
def test_norm_grad_strides(dev, n, pad):
    check_norm_grad(dev, 21, n, BF, SF, BF, BF, pad=pad, seed=2)
    check_norm_grad(dev, 21, n, HF, HF, HF, HF, pad=pad, seed=3)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [24, 1030])
def test_norm_grad_against_differences(dev, n):
    """sum(g y) along a direction: central differences in 64 bits."""
    gen = rng(8)
    g, h, w = rand(gen, 6, n), rand(gen, 6, n), 1 + rand(gen, n, std=0.2)
    gi, gw = fw.add_rms_norm_backward(g.to(dev), h.to(dev), w.to(dev))
    step = 1e-5
    f = lambda hh, ww: float((g.to(f64) * norm64(hh, None, ww, 1e-6)[1]).sum())  # noqa: E731
    for i in range(3):
        a, b = rand(gen, 6, n).to(f64), rand(gen, n).to(f64)
        dh = (f(h.to(f64) + step * a, w) - f(h.to(f64) - step * a, w)) / (2 * step)
        dw = (f(h.to(f64), w.to(f64) + step * b) - f(h.to(f64), w.to(f64) - step * b)) / (2 * step)
        # rounding of the gradient's values, and the differences' own error (step^2, 2^-53 / step of the sum's terms)
        terms = float((g.to(f64) * norm64(h, None, w, 1e-6)[1]).abs().sum())
        slack = 1e-8 * terms
        assert abs(float((gi.cpu().to(f64) * a).sum()) - dh) <= F * 4 * float((gi.cpu().to(f64) * a).abs().sum()) + slack
        assert abs(float((gw.cpu().to(f64) * b).sum()) - dw) <= F * 4 * float((gw.cpu().to(f64) * b).abs().sum()) + slack


# ---- the int8 product -------------------------------------------------------
def int8(gen, *shape):
    return torch.randint(-128, 128, shape, generator=gen, dtype=torch.int64).to(I8)


def mm_want(a, w, sa, sw, bias, out):
    """The definition, each binary32 step in turn: the sums are exact in float64."""
    acc = a.double() @ w.double().t()
    y = acc.float() * sa.reshape(-1, 1) * sw.reshape(1, -1)
    if bias is not None:
        y = y + bias.float()
    return y.to(out)


def check_mm(dev, M, N, K, out=BF, bias=None, per=(True, True), pad=(0, 0), seed=0, codes=None, pad_out=0):
    gen = rng(seed)
    a, w = codes or (int8(gen, M, K), int8(gen, N, K))
    sa = torch.rand(M, 1, generator=gen) * 0.05 + 0.01 if per[0] else torch.tensor([0.03])
    sw = torch.rand(1, N, generator=gen) * 2e-3 + 1e-4 if per[1] else torch.tensor([0.0011])
    b = None if bias is None else rand(gen, N, dtype=bias)
    note(f"int8 {M}x{N}x{K} {out} bias={bias} per={per} pad={pad}")
    ad, wd = (t.to(dev) if p == 0 else _wide8(t, p, dev) for t, p in zip((a, w), pad))
    o = None
    if pad_out:
        o = torch.full((M, N + pad_out), 5.0, dtype=out, device=dev)[:, 1:1 + N]
    y = fw.int8_scaled_mm(ad, wd.t(), sa.to(dev), sw.to(dev), bias=None if b is None else b.to(dev), out_dtype=out, out=o)
    torch.cuda.synchronize(dev)
    want = mm_want(a, w, sa, sw, b, out)
    bad = (y.cpu() != want).nonzero()
    assert y.shape == (M, N) and not len(bad), (len(bad), bad[:4].tolist())
    if pad_out:
        whole = o._base if o._base is not None else o
        assert (whole[:, 0] == 5).all() and (whole[:, 1 + N:] == 5).all()


def _wide8(t, pad, dev):
    big = torch.full((t.shape[0], t.shape[1] + pad), 99, dtype=I8)
    big[:, 1:1 + t.shape[1]] = t
    return big.to(dev)[:, 1:1 + t.shape[1]]


MM = [(1, 1, 1), (1, 16, 64), (1, 5760, 1920), (2, 100, 130), (3, 4096, 512), (7, 129, 65), (16, 64, 64), (17, 333, 1000),
      (31, 96, 4096), (33, 1000, 77), (64, 5760, 1920), (65, 65, 127), (100, 257, 513), (128, 128, 128), (130, 250, 1925),
      (250, 512, 4096), (256, 256, 256), (257, 300, 1024), (300, 700, 3000), (513, 1030, 640), (1024, 1024, 1040),
      (1, 300, 16384), (5, 40, 131071)]


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", MM)
@pytest.mark.parametrize("out,bias,per", [(BF, None, (True, True)), (HF, HF, (True, False)), (SF, SF, (False, True)),
                                          (BF, SF, (False, False))])
def test_int8_mm(dev, M, N, K, out, bias, per):
    check_mm(dev, M, N, K, out, bias, per)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(1, 200, 96), (20, 130, 100), (70, 64, 1000), (300, 310, 520), (600, 600, 1100)])
@pytest.mark.parametrize("pad", [(2, 0), (0, 3), (16, 16), (15, 17)])
def test_int8_mm_strides(dev, M, N, K, pad):
    check_mm(dev, M, N, K, pad=pad, seed=1, pad_out=3)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 40, 300])
def test_int8_mm_largest_sums(dev, M):
    """-128 x -128 all along the longest K: 2147467264, just inside int32."""
    K = 131071
    check_mm(dev, M, 48, K, SF, codes=(torch.full((M, K), -128, dtype=I8), torch.full((48, K), -128, dtype=I8)))


@pytest.mark.gpu
def test_int8_mm_empty(dev):
    one = torch.ones(1, device=dev)
    b = torch.arange(8, dtype=BF, device=dev)
    y = fw.int8_scaled_mm(torch.empty(3, 0, dtype=I8, device=dev), torch.empty(8, 0, dtype=I8, device=dev).t(), one, one,
                          bias=b)
    assert torch.equal(y, b.expand(3, 8))
    y = fw.int8_scaled_mm(torch.empty(0, 64, dtype=I8, device=dev), torch.empty(8, 64, dtype=I8, device=dev).t(), one, one)
    assert y.shape == (0, 8)


# ---- token log probabilities ------------------------------------------------
def logp64(z, tokens, k):
    z = z.to(f64)
    empty = (z == -INF).all(1)
    broken = z.isnan().any(1) | (z == INF).any(1)
    m = z.amax(1)
    log_sum = (z - m[:, None]).exp().sum(1).log()
    lse = torch.where(broken, math.nan, torch.where(empty, -INF, m + log_sum))
    lp = torch.where(empty[:, None], -INF, z - m[:, None] - log_sum[:, None])
    lp = torch.where(broken[:, None], math.nan, lp)
    p = lp.exp()
    ent = torch.where(p > 0, -p * lp, 0.0).sum(1)
    ent = torch.where(broken, math.nan, ent)
    size = torch.where(p > 0, p * lp.abs(), 0.0).sum(1)
    V = z.shape[1]
    got = lp.gather(1, tokens.clamp(0, V - 1))
    got = torch.where(tokens >= V, math.nan, torch.where(tokens < 0, 0.0, got))
    order = torch.sort(z + 0.0, dim=1, descending=True, stable=True).indices[:, :k]
    order = torch.where(z.isnan().any(1)[:, None], -1, order)
    top = torch.where(order < 0, math.nan, lp.gather(1, order.clamp_min(0)))
    return got, ent, lse, top, order, size


def check_logp(dev, z, tokens, k, pad=0):
    note(f"logprobs {tuple(z.shape)} {z.dtype} tokens {tuple(tokens.shape)} k={k} pad={pad}")
    r = fw.token_logprobs(wide(z, pad, dev), tokens.to(dev), top_k=k)
    torch.cuda.synchronize(dev)
    t2 = tokens if tokens.dim() == 2 else tokens[:, None]
    got, ent, lse, top, order, size = logp64(z, t2, k)
    fin = lambda t: t.abs().nan_to_num(nan=0.0, posinf=0.0)  # noqa: E731
    log_sum = fin(lse - z.to(f64).amax(1))
    tol_lse = F * (1 + fin(lse))
    close(r.lse, lse, tol_lse, "lse")
    # log S and U / S, each of up to the entropy and the largest log probability
    close(r.entropy, ent, F * (1 + 2 * log_sum + size), "entropy")
    close(r.logprobs.reshape(got.shape), got, tol_lse[:, None] + fin(got) * F, "logprobs")
    assert r.logprobs.shape == tokens.shape and r.entropy.shape == r.lse.shape == (z.shape[0],)
    if k:
        assert r.top_tokens.dtype == torch.int64
        assert torch.equal(r.top_tokens.cpu(), order), "top tokens"
        close(r.top_logprobs, top, tol_lse[:, None] + fin(top) * F, "top logprobs")
    else:
        assert r.top_logprobs is None and r.top_tokens is None
    return r


def make_logits(gen, T, V, dtype, masked=False):
    z = rand(gen, T, V, std=2.5, dtype=dtype)
    if masked:
        z = z.masked_fill(torch.rand(T, V, generator=gen) < 0.4, -INF)
    return z


LOGP = [(1, 1, 1), (1, 2, 2), (3, 5, 5), (2, 64, 20), (4, 100, 64), (1, 2047, 20), (2, 2048, 5), (2, 2049, 1), (5, 4096, 20),
        (1, 4097, 20), (3, 9001, 5), (1, 50257, 20), (1, 131072, 64), (7, 32001, 5), (600, 1000, 3), (520, 6000, 20),
        (40, 30000, 20)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,V,k", LOGP)
@pytest.mark.parametrize("dtype,C,masked", [(BF, 1, False), (HF, 4, True), (SF, 0, False), (SF, None, True)])
def test_logp(dev, T, V, k, dtype, C, masked):
    gen = rng(T * 7 + V)
    z = make_logits(gen, T, V, dtype, masked)
    tokens = torch.randint(-1, V, (T,) if C is None else (T, C), generator=gen)
    check_logp(dev, z, tokens, k)
    check_logp(dev, z, tokens, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("pad", [2, 3, 8])
@pytest.mark.parametrize("T,V", [(3, 50), (2, 5000), (515, 2051)])
def test_logp_strides(dev, T, V, pad):
    gen = rng(pad)
    check_logp(dev, make_logits(gen, T, V, BF), torch.randint(0, V, (T, 2), generator=gen), 4, pad=pad)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [2, 513])
@pytest.mark.parametrize("V", [40, 5000, 20000])
@pytest.mark.parametrize("k", [1, 20, 33])
def test_logp_crowded_top(dev, T, V, k):
    """Ties everywhere, the largest logits side by side in one thread's
    vectors, falling and rising rows, few distinct values."""
    idx = torch.arange(V)
    rows = [torch.zeros(V), -idx.float(), idx.float(), (idx % 3).float(), ((idx // 8) % 256 == 5).float() * 9 + (idx % 7) * 0.1,
            torch.where(idx % 2 == 0, 0.0, -0.0), torch.where(idx < 30, -INF, -3.4028234663852886e38),
            torch.where(idx % 8 == 7, -3.4028234663852886e38, -INF), torch.where(idx == V - 1, 1.0, -INF),
            ((idx // 8) % 256 < 2).float() * 5 + (idx % 11).float()]
    z = torch.stack([rows[i % len(rows)] for i in range(max(T, len(rows)) if T > 2 else len(rows))])
    tokens = torch.full((z.shape[0], 1), V - 1)
    check_logp(dev, z, tokens, min(k, V))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, HF, SF])
@pytest.mark.parametrize("T,V", [(8, 37), (8, 9000), (640, 3000)])
def test_logp_special_rows(dev, T, V, dtype):
    """Nothing but -inf, one logit left, masks of the type's lowest value,
    NaN, +inf, huge spans; tokens that are none, out of the vocabulary, masked."""
    z = rand(rng(9), T, V, std=2.0, dtype=dtype)
    low = torch.finfo(dtype).min
    z[0] = -INF
    z[1] = -INF
    z[1, V // 2] = 3.0
    z[2, 1:] = low
    z[3] = low
    z[4, V - 1] = math.nan
    z[5, 3] = INF
    z[6, ::2] = torch.finfo(dtype).max
    z[7] = -INF
    z[7, :2] = low
    tokens = torch.stack([torch.full((T,), -1), torch.full((T,), V), torch.zeros(T, dtype=torch.int64),
                          torch.full((T,), V // 2), torch.full((T,), -5), torch.full((T,), 1 << 40)], 1)
    check_logp(dev, z, tokens, 7)


@pytest.mark.gpu
def test_logp_far_rows(dev):
    """Row offsets beyond 2^31 elements: the last rows are right."""
    V = 1 << 20
    T = 2100
    z = torch.empty(T, V, dtype=BF, device=dev)
    z.fill_(-INF)
    last = rand(rng(3), 2, V, dtype=BF)
    z[-2:] = last.to(dev)
    tokens = torch.full((T,), 5, device=dev)
    r = fw.token_logprobs(z, tokens, top_k=3)
    got, ent, lse, top, order, _ = logp64(last, torch.full((2, 1), 5), 3)
    assert torch.equal(r.top_tokens[-2:].cpu(), order)
    close(r.logprobs[-2:], got[:, 0], F * (2 + 2 * lse.abs()), "logprobs")
    assert (r.lse[:-2] == -INF).all()
    d = fw.token_logprobs_backward(z, tokens, r.lse, r.entropy, torch.ones(T, device=dev), out=z)
    assert d.data_ptr() == z.data_ptr()
    want = -torch.softmax(last.to(f64), 1)
    want[:, 5] += 1
    close(d[-2:], want, half_step(want, BF) + F * want.abs(), "gradient")
    assert (d[:3] == 0).all()


# ---- their gradient ---------------------------------------------------------
def logp_grad64(z, tokens, lse, ent, g, ge, top, gtop):
    """The definition at the given lse and entropy; and the size of its terms."""
    z, V = z.to(f64), z.shape[1]
    d = z - lse.to(f64)[:, None]
    p = d.exp()
    lp = torch.where(z == -INF, 0.0, d)
    out, size = torch.zeros_like(z), torch.zeros_like(z)
    total = torch.zeros(z.shape[0], dtype=f64)
    broken = lse.isnan()
    for tok, val in ((tokens, g), (top, gtop)):
        if val is None:
            continue
        broken = broken | (tok >= V).any(1)
        val = torch.where(tok < 0, 0.0, val.to(f64))
        at = tok.clamp(0, V - 1)
        out.scatter_add_(1, at, val)
        size.scatter_add_(1, at, val.abs())
        total = total + val.sum(1)
        size = size + p * val.abs().sum(1, keepdim=True)
    out = out - p * total[:, None]
    if ge is not None:
        e = ge.to(f64)[:, None]
        out = out - e * p * (lp + ent.to(f64)[:, None])
        size = size + e.abs() * p * (lp.abs() + ent.to(f64).abs()[:, None])
    empty = lse == -INF
    out[empty], size[empty] = 0, 0
    out[broken] = math.nan
    return out, size * (1 + lp.abs())   # exp turns an error of lp into one of p


def check_logp_grad(dev, z, tokens, g, ge, top, gtop, pad=0, inplace=False):
    note(f"logprobs gradient {tuple(z.shape)} {z.dtype} C={tokens.shape[1]} top={None if top is None else top.shape[1]} pad={pad}")
    zd = wide(z, pad, dev)
    r = fw.token_logprobs(zd, tokens.to(dev))
    to = lambda t: None if t is None else t.to(dev)  # noqa: E731
    d = fw.token_logprobs_backward(zd, tokens.to(dev), r.lse, r.entropy, to(g), to(ge), top_tokens=to(top),
                                   grad_top=to(gtop), out=zd if inplace else None)
    torch.cuda.synchronize(dev)
    want, size = logp_grad64(z, tokens, r.lse.cpu(), r.entropy.cpu(), g, ge, top, gtop)
    assert d.dtype == z.dtype
    close(d, want, half_step(want.nan_to_num(nan=0.0), z.dtype) + F * size.nan_to_num(nan=0.0), "gradient")


@pytest.mark.gpu
@pytest.mark.parametrize("T,V", [(1, 1), (2, 7), (3, 64), (2, 2049), (3, 8192), (2, 8193), (5, 32001), (300, 1111)])
@pytest.mark.parametrize("dtype,C,k,ent", [(BF, 1, 0, True), (HF, 4, 5, False), (SF, 4, 5, True), (SF, 0, 0, True),
                                           (SF, 700, 20, True)])
@pytest.mark.parametrize("inplace", [False, True])
def test_logp_grad(dev, T, V, dtype, C, k, ent, inplace):
    gen = rng(V + C)
    z = make_logits(gen, T, V, dtype, masked=V > 7 and C == 4)
    if V > 7:
        z[:, 3] = 1.0
    tokens = torch.randint(-1, V, (T, C), generator=gen)
    top = torch.randint(0, V, (T, k), generator=gen) if k else None
    if C >= 4:
        tokens[:, 1] = tokens[:, 0]          # named twice, and again among the alternatives
        if k:
            top[:, 0] = tokens[:, 0].clamp_min(0)
    check_logp_grad(dev, z, tokens, rand(gen, T, C) if C else None, rand(gen, T) if ent else None, top,
                    rand(gen, T, k) if k else None, inplace=inplace)


@pytest.mark.gpu
@pytest.mark.parametrize("pad", [2, 3, 8])
@pytest.mark.parametrize("V", [50, 9001])
def test_logp_grad_strides(dev, V, pad):
    gen = rng(pad)
    check_logp_grad(dev, make_logits(gen, 4, V, BF), torch.randint(0, V, (4, 2), generator=gen), rand(gen, 4, 2),
                    rand(gen, 4), None, None, pad=pad)


@pytest.mark.gpu
def test_logp_grad_special_rows(dev):
    z = rand(rng(10), 5, 3001)
    z[0] = -INF
    z[1, 7] = math.nan
    z[2, 7] = INF
    z[3, 1:] = torch.finfo(SF).min
    tokens = torch.tensor([[5], [5], [5], [0], [3001]])
    check_logp_grad(dev, z, tokens, torch.ones(5, 1), torch.ones(5), None, None)


@pytest.mark.gpu
def test_logp_grad_against_differences(dev):
    gen = rng(11)
    T, V, C, k = 4, 300, 3, 4
    z = make_logits(gen, T, V, SF)
    tokens = torch.randint(0, V, (T, C), generator=gen)
    g, ge, gt = rand(gen, T, C), rand(gen, T), rand(gen, T, k)
    r = fw.token_logprobs(z.to(dev), tokens.to(dev), top_k=k)
    d = fw.token_logprobs_backward(z.to(dev), tokens.to(dev), r.lse, r.entropy, g.to(dev), ge.to(dev),
                                   top_tokens=r.top_tokens, grad_top=gt.to(dev)).cpu().to(f64)
    top = r.top_tokens.cpu()

    def loss(zz):
        lp = torch.log_softmax(zz, 1)
        ent = -(lp.exp() * lp).sum(1)
        return float((g * lp.gather(1, tokens)).sum() + (ge * ent).sum() + (gt * lp.gather(1, top)).sum())

    step = 1e-5
    for i in range(3):
        a = rand(gen, T, V).to(f64)
        diff = (loss(z.to(f64) + step * a) - loss(z.to(f64) - step * a)) / (2 * step)
        # the gradient's values are off by F of terms that p times up to (1 + |lp|) bounds
        assert abs(float((d * a).sum()) - diff) <= 20 * F * (float(g.abs().sum() + gt.abs().sum() + 10 * ge.abs().sum())) + 1e-6


@pytest.mark.gpu
def test_broadcast_gradients(dev):
    """Expanded gradients, as autograd's sums hand them on."""
    z = rand(rng(12), 6, 500).to(dev)
    tokens = torch.arange(6, device=dev)
    r = fw.token_logprobs(z, tokens)
    one = torch.ones(1, device=dev)
    a = fw.token_logprobs_backward(z, tokens, r.lse, r.entropy, one.expand(6), one.expand(6))
    b = fw.token_logprobs_backward(z, tokens, r.lse, r.entropy, one.repeat(6), one.repeat(6))
    assert torch.equal(a, b)


# ---- streams and graphs -----------------------------------------------------
@pytest.mark.gpu
def test_other_stream_and_graph(dev):
    """The same bits on another stream, and on every replay of a captured
    chain, with eager work between the replays."""
    gen = rng(13)
    x, res, w = rand(gen, 48, 1920, dtype=BF).to(dev), rand(gen, 48, 1920, dtype=BF).to(dev), torch.ones(1920, dtype=BF, device=dev)
    w8, sw = int8(gen, 5000, 1920).to(dev), torch.full((1, 5000), 1e-4, device=dev)
    tokens = torch.arange(48, device=dev)
    g = rand(gen, 48).to(dev)

    def chain():
        q, s, h = fw.add_rms_norm_quant(x, w, res, out_dtype=I8)
        z = fw.int8_scaled_mm(q, w8.t(), s, sw, out_dtype=SF)
        r = fw.token_logprobs(z, tokens, top_k=5)
        d = fw.token_logprobs_backward(z, tokens, r.lse, r.entropy, g, g)
        gi, gw = fw.add_rms_norm_backward(x, h, w, grad_h=res)
        return [q.float(), s, h, z, r.logprobs, r.entropy, r.top_tokens, d, gi, gw]

    eager = [t.clone() for t in chain()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = chain()
        chain()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(eager, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = chain()
    for i in range(3):
        for t in held:
            t.zero_()
        chain()
        graph.replay()
        torch.cuda.synchronize(dev)
        assert all(torch.equal(a, b) for a, b in zip(eager, held)), f"replay {i}"


# ---- refusals (no GPU: they fail before any call) ---------------------------
def c_norm(**kw):
    a = dict(x=16, xd=0, ldx=64, w=16, wd=0, res=None, rd=0, ldr=0, T=2, n=64, eps=1e-6, q=16, qd=3, ldq=64, scale=16,
             rows=None, h=None, ldh=0)
    a.update(kw)
    return operators._lib().emu_add_rms_norm_quant(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), 1), (dict(n=-1), 1), (dict(n=0, ldx=0, ldq=0), 1), (dict(xd=3), 1), (dict(xd=9), 1), (dict(wd=1), 1),
    (dict(qd=0), 1), (dict(qd=6), 1), (dict(x=None), 1), (dict(w=None), 1), (dict(q=None), 1), (dict(scale=None), 1),
    (dict(ldx=63), 1), (dict(ldq=63), 1), (dict(res=16, rd=1, ldr=64), 1), (dict(res=16, ldr=63), 1), (dict(h=16, ldh=64), 1),
    (dict(res=16, ldr=64, h=16, ldh=63), 1), (dict(eps=-1.0), 1), (dict(eps=math.nan), 1), (dict(x=17), 1),
    (dict(w=18, wd=2), 1), (dict(scale=18), 1), (dict(T=2 ** 31), 3), (dict(n=2 ** 30 + 1, ldx=2 ** 31, ldq=2 ** 31), 3),
    (dict(ldx=2 ** 62), 1), (dict(T=0), 0)])
def test_norm_refusals(kw, status):
    assert c_norm(**kw) == status
    assert bool(operators._lib().emu_last_error_message()) == (status != 0)


def c_norm_grad(**kw):
    a = dict(g=16, gd=0, ldg=64, h=16, hd=0, ldh=64, w=16, wd=0, gh=None, ghd=0, ldgh=0, T=2, n=64, eps=1e-6, gi=16, ldgi=64,
             gw=16, ws=16, wsb=1 << 20)
    a.update(kw)
    return operators._lib().emu_add_rms_norm_backward(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), 1), (dict(n=0), 1), (dict(gd=4), 1), (dict(hd=1), 1), (dict(wd=1), 1), (dict(gh=16, ghd=1, ldgh=64), 1),
    (dict(g=None), 1), (dict(h=None), 1), (dict(w=None), 1), (dict(gi=None), 1), (dict(gw=None), 1), (dict(ldg=1), 1),
    (dict(ldh=1), 1), (dict(ldgi=1), 1), (dict(gh=16, ldgh=1), 1), (dict(ws=None), 4), (dict(wsb=16), 4), (dict(ws=20), 1),
    (dict(h=18, hd=2), 1), (dict(T=2 ** 31), 3)])
def test_norm_grad_refusals(kw, status):
    assert c_norm_grad(**kw) == status


def c_mm(**kw):
    a = dict(a=16, lda=64, w=16, ldw=64, M=4, N=32, K=64, sa=16, pa=1, sw=16, pw=1, bias=None, bd=0, out=16, od=0, ldo=32,
             ws=16, wsb=1 << 30)
    a.update(kw)
    return operators._lib().emu_int8_scaled_mm(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), 1), (dict(K=-1), 1), (dict(od=3), 1), (dict(od=5), 1), (dict(bias=16, bd=1), 1), (dict(a=None), 1),
    (dict(w=None), 1), (dict(out=None), 1), (dict(sa=None), 1), (dict(sw=None), 1), (dict(lda=63), 1), (dict(ldw=63), 1),
    (dict(ldo=31), 1), (dict(out=17), 1), (dict(sa=18), 1), (dict(bias=18, bd=2), 1), (dict(K=131072, lda=131072, ldw=131072), 3),
    (dict(M=2 ** 31), 3), (dict(M=0), 0), (dict(N=0), 0)])
def test_int8_mm_refusals(kw, status):
    assert c_mm(**kw) == status


def c_logp(**kw):
    a = dict(z=16, zd=0, ldz=100, T=2, V=100, tok=16, C=1, k=5, lp=16, ent=16, lse=16, tlp=16, tt=16, ws=16, wsb=1 << 20)
    a.update(kw)
    return operators._lib().emu_token_logprobs(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), 1), (dict(V=0), 1), (dict(C=-1), 1), (dict(k=-1), 1), (dict(zd=3), 1), (dict(z=None), 1), (dict(tok=None), 1),
    (dict(lp=None), 1), (dict(ent=None), 1), (dict(lse=None), 1), (dict(tlp=None), 1), (dict(tt=None), 1), (dict(ldz=99), 1),
    (dict(k=101), 3), (dict(V=50, ldz=50, k=51), 1), (dict(k=65), 3), (dict(tok=20), 1), (dict(z=17), 1), (dict(T=2 ** 31), 3),
    (dict(V=2 ** 31, ldz=2 ** 31), 3), (dict(V=100000, ldz=100000, ws=None), 4), (dict(V=100000, ldz=100000, wsb=8), 4),
    (dict(ws=8), 1), (dict(T=0), 0)])
def test_logp_refusals(kw, status):
    assert c_logp(**kw) == status


def c_logp_grad(**kw):
    a = dict(z=16, zd=0, ldz=100, T=2, V=100, tok=16, C=1, lse=16, ent=16, g=16, ge=16, top=None, gtop=None, k=0, out=16, ldo=100)
    a.update(kw)
    return operators._lib().emu_token_logprobs_backward(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), 1), (dict(zd=5), 1), (dict(z=None), 1), (dict(lse=None), 1), (dict(out=None), 1), (dict(tok=None), 1),
    (dict(ent=None), 1), (dict(gtop=16, k=3), 1), (dict(ldz=99), 1), (dict(ldo=99), 1), (dict(C=1025), 3),
    (dict(C=1000, top=16, gtop=16, k=25), 3), (dict(T=0), 0), (dict(V=0), 0)])
def test_logp_grad_refusals(kw, status):
    assert c_logp_grad(**kw) == status


def test_workspaces():
    lib = operators._lib()
    assert lib.emu_add_rms_norm_backward_workspace(0, 64) == 0 and lib.emu_add_rms_norm_backward_workspace(-1, 64) == 0
    assert lib.emu_add_rms_norm_backward_workspace(1, 2048) == 2048 * 4
    assert lib.emu_token_logprobs_workspace(4096, 131072, 20) == 0      # a workgroup a row
    assert lib.emu_token_logprobs_workspace(1, 50257, 20) > 0
    assert lib.emu_token_logprobs_workspace(1, 50257, 65) == 0
    assert lib.emu_int8_scaled_mm_workspace(-1, 64, 64, 1) == 0 and lib.emu_int8_scaled_mm_workspace(4, 64, 131072, 1) == 0


def test_host_tensors_and_types_are_refused():
    x, w = torch.zeros(2, 64), torch.ones(64)
    with pytest.raises(ValueError):
        fw.add_rms_norm_quant(x, w)
    with pytest.raises(ValueError):
        fw.add_rms_norm_backward(x, x, w)
    with pytest.raises(ValueError):
        fw.int8_scaled_mm(torch.zeros(2, 64, dtype=I8), torch.zeros(8, 64, dtype=I8).t(), w[:1], w[:1])
    with pytest.raises(TypeError):
        fw.int8_scaled_mm(x, x.t(), w[:1], w[:1])
    with pytest.raises(ValueError):
        fw.token_logprobs(x, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError):
        fw.token_logprobs_backward(x, torch.zeros(2, dtype=torch.int64), x[:, 0], x[:, 0])


@pytest.mark.gpu
def test_binding_refusals(dev):
    x, w = torch.zeros(4, 64, device=dev), torch.ones(64, device=dev)
    i = torch.zeros(4, 64, dtype=I8, device=dev)
    tok = torch.zeros(4, dtype=torch.int64, device=dev)
    for bad in (lambda: fw.add_rms_norm_quant(x.t(), w[:4]), lambda: fw.add_rms_norm_quant(x, w[:32]),
                lambda: fw.add_rms_norm_quant(x, w, x[:2]), lambda: fw.add_rms_norm_quant(x, w, h_out=x),
                lambda: fw.add_rms_norm_quant(x, w, scale=w), lambda: fw.add_rms_norm_backward(x, x[:2], w),
                lambda: fw.add_rms_norm_quant(x, w, x.cpu()), lambda: fw.int8_scaled_mm(i, i.t(), w, w[:1]),
                lambda: fw.int8_scaled_mm(i, i, w[:1], w[:1]), lambda: fw.int8_scaled_mm(i, i.t(), w[:4], w[:1].double()),
                lambda: fw.int8_scaled_mm(i, i.t(), w[:1], w[:1], bias=w), lambda: fw.token_logprobs(x, tok[:3]),
                lambda: fw.token_logprobs(x, tok.cpu()), lambda: fw.token_logprobs_backward(x, tok, x[0], x[0]),
                lambda: fw.token_logprobs_backward(x, tok, x[:, 0], None, grad_entropy=x[:, 0])):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: fw.add_rms_norm_quant(x.double(), w), lambda: fw.add_rms_norm_quant(x.half(), w.bfloat16()),
                lambda: fw.token_logprobs(x, tok.int()), lambda: fw.add_rms_norm_backward(x, x.half(), w)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: fw.add_rms_norm_quant(x, w, out_dtype=BF), lambda: fw.int8_scaled_mm(i, i.t(), w[:1], w[:1], out_dtype=E4),
                lambda: fw.token_logprobs(x, tok, top_k=65), lambda: fw.token_logprobs(x[:, :5], tok, top_k=6)):
        with pytest.raises(fw.EmuError):
            bad()
    with pytest.raises(RuntimeError):
        fw.token_logprobs(x.clone().requires_grad_(), tok)
    with torch.no_grad():
        fw.token_logprobs(x.clone().requires_grad_(), tok)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(260, 260, 16), (513, 390, 1360), (1024, 8192, 384), (2048, 2048, 272), (3000, 3000, 512),
                                   (100, 100, 16384), (129, 70, 8208), (2100, 2300, 1000), (2300, 2100, 1111)])
def test_int8_mm_tiles(dev, M, N, K):
    """Every tile, whole and ragged, a split of K, stages that end within K."""
    check_mm(dev, M, N, K, BF, SF, seed=3)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(2 ** 18 + 5, 33, 16), (2 ** 18 + 70, 20, 33), (3, 2 ** 20 + 3, 16), (70, 2 ** 20 + 65, 16)])
def test_int8_mm_slices(dev, M, N, K):
    """More rows or columns than one launch takes."""
    check_mm(dev, M, N, K, HF, HF, seed=4)


@pytest.mark.gpu
def test_int8_mm_wide_rows(dev):
    """Leading dimensions beyond the tiles' 31-bit offsets: rows laid out anew."""
    big = torch.zeros(300, 1 << 23, dtype=I8, device=dev)
    gen = rng(5)
    a, w = int8(gen, 300, 512), int8(gen, 200, 512)
    big[:, 64:576] = a.to(dev)
    sa = torch.full((1,), 0.01, device=dev)
    y = fw.int8_scaled_mm(big[:, 64:576], w.to(dev).t(), sa, sa, out_dtype=SF)
    assert torch.equal(y.cpu(), mm_want(a, w, sa.cpu(), sa.cpu(), None, SF))


@pytest.mark.gpu
def test_leading_axes_and_argument_types(dev):
    """Rows of several axes are one axis of rows with one stride, or refused;
    arguments of other kinds are refused by name."""
    base = torch.zeros(4, 6, 64, device=dev)
    w = torch.ones(64, device=dev)
    for x in (base, base[:, :1], base[1:2], base.view(2, 2, 6, 64), base[::2, 0], base[:0], base[:, 3]):
        codes, scale, _ = fw.add_rms_norm_quant(x, w)
        assert codes.shape == x.shape and scale.shape == x.shape[:-1] + (1,)
    for x in (base[:, :3], base.transpose(0, 1), base[::2, ::2]):
        with pytest.raises(ValueError, match="one axis of rows"):
            fw.add_rms_norm_quant(x, w)
    with pytest.raises(ValueError, match="at least one axis"):
        fw.add_rms_norm_quant(w[0], w)
    tok = torch.zeros(4, dtype=torch.int64, device=dev)
    for bad in (lambda: fw.add_rms_norm_quant(base, 1.0), lambda: fw.add_rms_norm_quant(base, w, eps="small"),
                lambda: fw.token_logprobs(base[0], [0] * 6), lambda: fw.token_logprobs(base[0, :4], tok, top_k=1.5),
                lambda: fw.int8_scaled_mm(None, None, w, w)):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(fw.EmuError) as e:
        fw.token_logprobs(base[0, :4], tok, top_k=-1)
    assert e.value.status == 1
    with pytest.raises(fw.EmuError) as e:
        fw.add_rms_norm_quant(base, w, out_dtype="int8")
    assert e.value.status == 3


# ---- all of them together ---------------------------------------------------
@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["int8", "fp8"])
@pytest.mark.parametrize("T,n,V", [(1, 64, 96), (33, 192, 500)])
def test_policy_step(dev, kind, T, n, V):
    """A step's loss and gradients against autograd in 64 bits, from the step's own codes."""
    from bit_exact_fp8_amd import policy_step as ps
    note(f"policy step {kind} T={T} n={n} V={V}")
    gen = rng(T + n)
    V -= V % 16
    weight = rand(gen, V, n, std=n ** -0.5)
    branch, stream, nw = rand(gen, T, n), rand(gen, T, n), 1 + rand(gen, n, std=0.1)
    tokens, adv = torch.randint(0, V, (T,), generator=gen), rand(gen, T)
    other = rand(gen, T, n, std=1e-3)
    head = ps.int8_head(weight.to(dev)) if kind == "int8" else ps.fp8_head(weight.to(dev), 1 / 32)
    s = ps.policy_step(branch.to(dev), stream.to(dev), nw.to(dev), head, tokens.to(dev), adv.to(dev), 0.05,
                       grad_stream=other.to(dev))
    codes, scale, _ = fw.add_rms_norm_quant(branch.to(dev), nw.to(dev), stream.to(dev), out_dtype=I8 if kind == "int8" else E4,
                                            scale=head.in_scale)
    W = head.weight().cpu().to(f64)
    if kind == "int8":
        z = (codes.float() * scale).cpu().to(f64) @ W.t()
    else:  # (the emulated product's own values: it cuts its sums)
        z = fw.scaled_mm(codes, head.codes.t(), scale, head.scale, out_dtype=SF, use_fast_accum=True).cpu().to(f64)
    z.requires_grad_()
    lp = torch.log_softmax(z, 1)
    ent = -(lp.exp() * lp).sum(1)
    loss = -(adv.to(f64) * lp.gather(1, tokens[:, None])[:, 0] + 0.05 * ent).mean()
    loss.backward()
    h = (branch.to(f64) + stream.to(f64)).requires_grad_()
    w = nw.to(f64).requires_grad_()
    y = h / (h.pow(2).mean(1, keepdim=True) + 1e-6).sqrt() * w
    dy = z.grad @ W
    y.backward(dy)
    # logits of some 4 with errors of F (1 + |z|); p and its gradient follow
    # them, and the sums over V and n add their terms' absolute values
    zmax = 1 + z.detach().abs().amax()
    dz = F * 4 * zmax * (z.grad.abs() + adv.to(f64).abs().max() / T * lp.detach().exp())
    ddy = dz @ W.abs() + F * (z.grad.abs() @ W.abs())
    r = (h.detach().pow(2).mean(1, keepdim=True) + 1e-6).rsqrt()
    u, nv = dy.abs() * w.detach().abs(), h.detach().abs() * r
    du = ddy * w.detach().abs() + F * u
    dh = r * (du + nv * (du * nv).mean(1, keepdim=True) + F * nv * (u * nv).mean(1, keepdim=True))
    close(s.loss[None], loss.detach()[None], (F * 4 * zmax * (1 + adv.to(f64).abs().mean()) * 10)[None], "loss")
    close(s.grad_stream, h.grad + other.to(f64), dh + F * (h.grad.abs() + other.to(f64).abs()), "stream's gradient")
    close(s.grad_weight, w.grad, (ddy * nv + F * dy.abs() * nv).sum(0), "weight's gradient")


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["int8", "fp8"])
def test_policy_step_learns(dev, kind):
    from bit_exact_fp8_amd import policy_step as ps
    assert ps.main(["--head", kind, "--steps", "1"]) > 2 * ps.main(["--head", kind, "--steps", "12"])


@pytest.mark.gpu
@pytest.mark.parametrize("out", [E4, E5, I8])
@pytest.mark.parametrize("n", [512, 1920, 8192, 20000])
def test_norm_codes_are_the_nearest(dev, out, n):
    """Codes of values that lie at and next to the borders between two: with
    ones and minus ones r is known, and a weight of a border's value (and its
    neighbours in binary32) puts y there.  The oracle is exact but for r's 2^-50."""
    q, r = MOST[out], 1 / math.sqrt(1 + 0.25)
    v = torch.ones(4, n)
    v[:, ::3] = -1
    grid = torch.arange(1, 127, dtype=f64) + 0.5 if out == I8 else None
    if grid is None:
        codes = torch.arange(1, 256, dtype=torch.uint8).view(out).to(f64)
        codes = codes[codes.isfinite() & (codes > 2.0 ** -9)].sort().values
        grid = (codes[1:] + codes[:-1]) / 2
    border = grid[torch.arange(n) % len(grid)]
    w = (border / r).to(SF)
    step = torch.tensor([-2, -1, 0, 1, 2])[(torch.arange(n) // len(grid)) % 5].to(torch.int32)
    w = (w.view(torch.int32) + step).view(SF)
    one = torch.ones(1)
    note(f"norm codes {out} n={n}")
    codes, _, _ = fw.add_rms_norm_quant(v.to(dev), w.to(dev), eps=0.25, out_dtype=out, scale=one.to(dev))
    y = (v.to(f64) * r * w.to(f64)).clamp(-q, q)
    got = codes.cpu().to(f64)
    # none of the type's values is nearer than the code
    if out == I8:
        near = (y - y.round()).abs()
    else:
        values = torch.arange(0, 256, dtype=torch.uint8).view(out).to(f64)
        values = values[values.isfinite()].sort().values.unique()
        at = torch.searchsorted(values, y.contiguous()).clamp(1, len(values) - 1)
        near = torch.minimum((values[at] - y).abs(), (values[at - 1] - y).abs())
    off = (got - y).abs() - near
    assert float((off / y.abs()).max()) <= 2.0 ** -46, float((off / y.abs()).max())
