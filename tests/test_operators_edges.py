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
from test_operators import check_logp_grad

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
    i8, row, tok = torch.zeros(16, 64, dtype=torch.int8, device=dev), torch.zeros(16, device=dev), torch.zeros(16, dtype=torch.int64, device=dev)
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
