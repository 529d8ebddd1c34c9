"""What tests/test_operators.py leaves of include/emu_operators.h: the
alignment that the kernels' memory accesses claim, refusals of what autograd
would lose, and the paths that only large or unusual calls take."""
import math
import os
import re
import subprocess

import pytest
import torch

import bit_exact_fp8_amd as fw
from bit_exact_fp8_amd import api, build, operators
from test_operators import (BF, E4, E5, F, HF, I8, MOST, SF, check_logp, check_logp_grad, check_norm, check_norm_grad, close,
                            f64, half_step, make_logits, norm64, rand, rng)

ELEMENT = {"float": 4, "half": 2, "bfloat": 2}


@pytest.mark.skipif(not os.path.exists(build.HIPCC), reason="no hipcc")
@pytest.mark.parametrize("source", ["emu_norm.hip", "emu_logprobs.hip"])
def test_rows_are_accessed_with_their_elements_alignment(source, tmp_path):
    """Rows begin at any element, so a vector of 8 of a row's elements is read
    and written with the element's alignment: what the compiler is told, in
    its own intermediate form of the kernels."""
    out = tmp_path / "kernels.ll"
    subprocess.run([build.HIPCC, *build.FLAGS, "--cuda-device-only", "-S", "-emit-llvm", os.path.join(build.CSRC, source),
                    "-o", str(out)], check=True, capture_output=True)
    seen, wrong = {"load": 0, "store": 0}, []
    for line in out.read_text().splitlines():
        if not (m := re.search(r"\b(load|store) <8 x (float|half|bfloat)>.* addrspace\(1\).*, align (\d+)", line)):
            continue
        seen[m[1]] += 1
        if int(m[3]) > ELEMENT[m[2]]:
            wrong.append(line.strip())
    assert min(seen.values()) > 0
    assert not wrong, (len(wrong), wrong[:3])


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


@pytest.mark.gpu
@pytest.mark.parametrize("out", [torch.float8_e4m3fn, torch.float8_e5m2, torch.int8])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n", [40, 2000, 20000])
def test_norm_rows_whose_squares_overflow(dev, n, dtype, out):
    """Finite values beyond 1.8e19 have an infinite mean and y = 0, also where
    a value times its weight is beyond binary32; an infinity stays NaN."""
    x = torch.full((3, n), 3e38, device=dev).to(dtype)
    x[1, ::2] = -1e30
    x[2, n // 2] = math.inf
    w = torch.full((n,), 2.0, device=dev, dtype=dtype)
    print(f"[gpu] norm of overflowing squares {n} {dtype} {out}", flush=True)
    codes, scale, _ = fw.add_rms_norm_quant(x, w, out_dtype=out)
    assert (codes[:2].float() == 0).all() and (scale[:2] == 2.0 ** -126).all() and scale[2].isnan()
    codes, _, _ = fw.add_rms_norm_quant(x, w, out_dtype=out, scale=torch.tensor([0.01], device=dev))
    codes = codes.float()
    assert (codes[:2] == 0).all()
    here = torch.arange(n, device=dev) == n // 2
    assert (codes[2, ~here] == 0).all() and (codes[2, n // 2] == 0 if out == torch.int8 else codes[2, n // 2].isnan())


# ---- autograd: what a call would lose is refused (no GPU: before any other check) ----
def calls_of(make):
    """Every call with make() in the place of each of its floating arguments in turn, by name."""
    z, w, one = torch.zeros(4, 64), torch.ones(64), torch.ones(1)
    i8, tok, row = torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4, dtype=torch.int64), torch.zeros(4)
    top = torch.zeros(4, 2, dtype=torch.int64)
    calls = [
        (fw.add_rms_norm_quant, dict(x=z, weight=w, residual=z, scale=one, h_out=z), ()),
        (fw.add_rms_norm_backward, dict(g=z, h=z, weight=w, grad_h=z), ()),
        (fw.int8_scaled_mm, dict(scale_a=one, scale_b=one, bias=w, out=torch.zeros(4, 64)),
         dict(mat1=i8, mat2=torch.zeros(64, 64, dtype=torch.int8).t(), out_dtype=torch.float32)),
        (fw.token_logprobs, dict(logits=z), dict(tokens=tok)),
        (fw.token_logprobs_backward, dict(logits=z, lse=row, entropy=row, grad_logprobs=row, grad_entropy=row,
                                          grad_top=torch.zeros(4, 2), out=z), dict(tokens=tok, top_tokens=top)),
    ]
    for call, floats, others in calls:
        for name in floats:
            yield f"{call.__name__}({name})", lambda: call(**{**floats, name: make(floats[name])}, **dict(others))


def test_gradients_that_would_be_lost_are_refused():
    for name, call in calls_of(lambda t: t.clone().requires_grad_()):
        with pytest.raises(RuntimeError, match="requires a gradient"):
            call()
            pytest.fail(name)
        with torch.no_grad(), pytest.raises((ValueError, TypeError)):  # (host tensors)
            call()


def test_tangents_that_would_be_lost_are_refused():
    from torch.autograd import forward_ad
    with forward_ad.dual_level():
        for name, call in calls_of(lambda t: forward_ad.make_dual(t.clone(), torch.ones_like(t))):
            with torch.no_grad(), pytest.raises(RuntimeError, match="tangent"):
                call()
                pytest.fail(name)


# ---- outputs that are given: autograd is told that they were written -----------
def writers(dev):
    """(name, a tensor to write, the call that does)"""
    z, w, one = torch.zeros(16, 64, device=dev), torch.ones(64, device=dev), torch.ones(1, device=dev)
    i8, row = torch.zeros(16, 64, dtype=torch.int8, device=dev), torch.zeros(16, device=dev)
    tok = torch.zeros(16, dtype=torch.int64, device=dev)
    f8 = i8.view(torch.float8_e4m3fn)
    yield "h_out", z.clone(), lambda t: fw.add_rms_norm_quant(z, w, t, h_out=t)
    yield "int8 out", z.clone()[:, :16], lambda t: fw.int8_scaled_mm(i8, i8.t(), one, one, out_dtype=torch.float32, out=t)
    yield "gradient's out", z.clone(), lambda t: fw.token_logprobs_backward(t, tok, row, row, row, out=t)
    yield "fp8 out", z.clone()[:, :16], lambda t: fw.scaled_mm(f8, f8.t(), one, one, out_dtype=torch.float32, out=t)
    yield "fp8 out, no allocation", z.clone()[:, :16], lambda t: api.scaled_mm_noalloc(f8, f8.t(), one, one, t)


@pytest.mark.gpu
def test_written_outputs_count_a_version(dev):
    for name, t, call in writers(dev):
        print(f"[gpu] {name}", flush=True)
        version = t._version
        call(t)
        assert t._version == version + 1, name
        # what autograd has saved of it is noticed at the backward pass
        leaf = torch.ones(t.shape, device=dev, requires_grad=True)
        y = (leaf * t).sum()
        with torch.no_grad():
            call(t)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.backward()
        version = t._version
        with pytest.raises((ValueError, TypeError, RuntimeError)):
            call(t[:, ::2])
        assert t._version == version, name
        with torch.inference_mode():  # such a tensor has no version, and autograd saves none
            u = t.clone()
            call(u)
        call(u)


# ---- token log probabilities ------------------------------------------------
@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [50, 9001])
def test_tokens_out_of_the_vocabulary_give_nan_in_empty_rows_too(dev, V, dtype):
    """A row of nothing but -inf has the gradient 0, but a token (or top token)
    of V or more gives its row NaN, whatever the logits."""
    z = torch.full((5, V), -math.inf, dtype=dtype)
    tokens = torch.tensor([[2, V], [2, V - 1], [-1, 1 << 40], [2, 2], [-1, -1]])
    top = torch.tensor([[1], [V], [1], [1], [0]])
    ones = torch.ones(5, 2)
    check_logp_grad(dev, z, tokens, ones, torch.ones(5), top, ones[:, :1])
    check_logp_grad(dev, z, tokens, ones * math.inf, None, None, None)


def test_limits_are_the_headers():
    """The limits that Python names are the header's, and where the calls refuse."""
    with open(os.path.join(build.ROOT, "include", "emu_operators.h")) as f:
        named = dict(re.findall(r"#define EMU_(MAX_\w+) (\d+)\n", f.read()))
    assert named == {"MAX_TOP_TOKENS": str(operators.MAX_TOP_TOKENS), "MAX_GRAD_TOKENS": str(operators.MAX_GRAD_TOKENS)}
    lib, most = operators._lib(), operators.MAX_GRAD_TOKENS
    for C, k, status in ((most, 0, 0), (most + 1, 0, 3), (most - 64, 64, 0), (most - 63, 64, 3)):
        assert lib.emu_token_logprobs_backward(16, 0, 100, 0, 100, 16, C, 16, None, 16, None, 16, 16 if k else None, k, 16, 100,
                                               None) == status
    assert lib.emu_token_logprobs_backward(16, 0, 100, 0, 100, 16, most + 1, 16, 16, None, 16, None, None, 0, 16, 100, None) == 0
    for k, status in ((operators.MAX_TOP_TOKENS, 0), (operators.MAX_TOP_TOKENS + 1, 3)):
        assert lib.emu_token_logprobs(16, 0, 100, 0, 100, 16, 1, k, 16, 16, 16, 16, 16, None, 0, None) == status


# ---- paths that only large or unusual calls take -----------------------------
@pytest.mark.gpu
@pytest.mark.parametrize("T,n,x_t,r_t,out,given", [(14001, 2057, BF, BF, E4, True), (4501, 4071, BF, SF, I8, False),
                                                   (26003, 801, SF, SF, E5, False), (3001, 9001, HF, SF, E4, True)])
def test_norm_past_the_cache(dev, T, n, x_t, r_t, out, given):
    """Calls of more than 192 MiB, which pass by the last-level cache."""
    check_norm(dev, T, n, x_t, r_t, out, given)


@pytest.mark.gpu
@pytest.mark.parametrize("T,n,g_t,h_t,gh_t", [(9001, 2807, BF, BF, BF), (3501, 3607, SF, SF, SF), (24001, 701, HF, SF, SF),
                                              (1801, 9007, BF, SF, SF)])
def test_norm_grad_past_the_cache(dev, T, n, g_t, h_t, gh_t):
    check_norm_grad(dev, T, n, g_t, h_t, gh_t, g_t)


@pytest.mark.gpu
@pytest.mark.parametrize("T,V,dtype,k", [(3301, 30503, HF, 0), (2003, 26003, SF, 0), (1501, 34001, SF, 4)])
def test_logp_past_the_cache(dev, T, V, dtype, k):
    gen = rng(V)
    z, tokens = make_logits(gen, T, V, dtype), torch.randint(-1, V, (T, 1), generator=gen)
    at = "cpu" if k else dev  # (where the definition is computed)
    check_logp(dev, z.to(at), tokens.to(at), k)


@pytest.mark.gpu
@pytest.mark.parametrize("T,V,dtype", [(1701, 30503, HF), (1003, 26003, SF)])
def test_logp_grad_past_the_cache(dev, T, V, dtype):
    gen = rng(V)
    z, tokens = make_logits(gen, T, V, dtype), torch.randint(-1, V, (T, 1), generator=gen)
    check_logp_grad(dev, z, tokens, rand(gen, T, 1), rand(gen, T), None, None, inplace=True)


@pytest.mark.gpu
@pytest.mark.parametrize("n,pad", [(3, 0), (9, 3)])
def test_norm_of_more_rows_than_a_launch(dev, n, pad):
    check_norm(dev, 2 ** 20 + 3, n, BF, SF, I8, False, pad=pad)
    check_norm(dev, 2 ** 20 + 3, n, HF, None, E4, True, pad=pad)


@pytest.mark.gpu
def test_logp_of_more_rows_than_a_launch(dev):
    gen = rng(20)
    T = 2 ** 20 + 3
    check_logp(dev, make_logits(gen, T, 5, BF), torch.randint(-1, 6, (T, 2), generator=gen), 2, pad=2)
    T = 2 ** 23 + 3
    check_logp_grad(dev, make_logits(gen, T, 2, HF), torch.randint(-1, 2, (T, 1), generator=gen), rand(gen, T, 1), None, None, None)


@pytest.mark.gpu
@pytest.mark.parametrize("T,V,k", [(3, 5000, 3), (2, 50001, 0), (513, 700, 2)])
def test_logp_of_more_tokens_than_threads(dev, T, V, k):
    """More than 256 tokens a row, of rows that are split and of whole ones."""
    gen = rng(V)
    check_logp(dev, make_logits(gen, T, V, SF), torch.randint(-1, V + 1, (T, 700), generator=gen), k)


@pytest.mark.gpu
@pytest.mark.parametrize("where", ["g", "grad_h"])
@pytest.mark.parametrize("T,n", [(5, 5), (40, 77), (700, 1925), (9, 9000), (3, 12001), (300, 17003)])
@pytest.mark.parametrize("dtype", [BF, SF])
def test_norm_grad_in_place(dev, T, n, dtype, where):
    """grad_in may be g or grad_h itself: the same bits as into another tensor."""
    gen = rng(n)
    g, h, gh = (rand(gen, T, n + 1, dtype=dtype).to(dev) for _ in range(3))
    w = rand(gen, n, dtype=dtype).to(dev)
    print(f"[gpu] norm gradient in place of {where} {T}x{n} {dtype}", flush=True)
    want, want_w = fw.add_rms_norm_backward(g[:, :n], h[:, :n], w, grad_h=gh[:, :n])
    lib, code, ld = operators._lib(), 0 if dtype == BF else 2, n + 1
    out, grad_w = (g if where == "g" else gh), torch.empty_like(w)
    need = lib.emu_add_rms_norm_backward_workspace(T, n)
    ws = torch.empty(need, dtype=torch.uint8, device=dev)
    status = lib.emu_add_rms_norm_backward(g.data_ptr(), code, ld, h.data_ptr(), code, ld, w.data_ptr(), code, gh.data_ptr(), code,
                                           ld, T, n, 1e-6, out.data_ptr(), ld, grad_w.data_ptr(), ws.data_ptr(), need,
                                           torch.cuda.current_stream(dev).cuda_stream)
    torch.cuda.synchronize(dev)
    assert status == 0 and torch.equal(out[:, :n], want) and torch.equal(grad_w, want_w)


@pytest.mark.gpu
@pytest.mark.parametrize("out", [E4, E5, I8])
@pytest.mark.parametrize("n", [40, 2000, 20000])
@pytest.mark.parametrize("given", [None, 2.0 ** -118, 2.0 ** -125])
def test_norm_of_very_small_weights(dev, n, out, given):
    """Scales under 2^-100.  y is made by two products in binary32, which near
    2^-126 are off by up to 2^-150 each whatever their size."""
    gen = rng(n)
    x = rand(gen, 4, n)
    w = (1 + torch.rand(n, generator=gen)) * torch.exp2(-112 - torch.randint(0, 20, (n,), generator=gen).float())
    w[0] = 2.0 ** -111
    x[:, 0] = 2.0
    print(f"[gpu] norm of small weights {n} {out} given={given}", flush=True)
    codes, scale, _ = fw.add_rms_norm_quant(x.to(dev), w.to(dev), out_dtype=out,
                                            scale=None if given is None else torch.tensor([given], device=dev))
    _, y = norm64(x, None, w, 1e-6)
    if given is None:
        want = (y.abs().amax(1, keepdim=True) / MOST[out]).clamp_min(2.0 ** -126)
        assert float(want.max()) < 2.0 ** -100
        # (three products and a quotient, the first of them possibly below 2^-126)
        close(scale, want, want * F, "scale")
    s = scale.cpu().to(f64)
    z = (y / s).clamp(-MOST[out], MOST[out])
    step = torch.full_like(z, 0.5) if out == I8 else half_step(z, out)
    close(codes.cpu().float(), z, step + z.abs() * F + 2.0 ** -149 / s, "codes")
