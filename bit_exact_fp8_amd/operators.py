"""The operators beside the FP8 product (C ABI in ``include/emu_operators.h``).

``add_rms_norm_quant`` / ``add_rms_norm_backward``: the residual's addition
with the RMS norm and 8-bit codes, and its gradient.  ``int8_scaled_mm``: the
product of 8-bit integers with scales per token and channel.
``token_logprobs`` / ``token_logprobs_backward``: log probabilities of given
tokens with entropy and top alternatives, and their gradient.

As in ``api``: argument checks and marshalling only, every step runs in the
HIP library's kernels on torch's current stream of the operands' device, and
there is no CPU fallback.  Calls take no part in autograd: the backward calls
are the caller's to make, and an input that requires a gradient is refused
while gradients are enabled.
"""
from __future__ import annotations

import ctypes
import math
from typing import NamedTuple

import torch

from . import api
from .api import EMU_ERR_UNSUPPORTED, EmuError, _check, _on_device, _operands

DTYPE = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2, torch.float8_e4m3fn: 3, torch.float8_e5m2: 4,
         torch.int8: 5}
QUANT_DTYPES = (torch.float8_e4m3fn, torch.float8_e5m2, torch.int8)
FLOAT_DTYPES = (torch.bfloat16, torch.float16, torch.float32)
MAX_TOP_TOKENS = 64          # EMU_MAX_TOP_TOKENS
INT8_MAX_ALIGNED_LD = 1 << 22   # EMU_INT8_MAX_ALIGNED_LD

_LIB = None


def _lib():
    global _LIB
    if _LIB is None:
        lib = api._lib()
        vp, i64, i32, f32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        lib.emu_add_rms_norm_quant.argtypes = [vp, i32, i64, vp, i32, vp, i32, i64, i64, i64, f32, vp, i32, i64, vp, vp,
                                               vp, i64, vp]
        lib.emu_add_rms_norm_backward.argtypes = [vp, i32, i64, vp, i32, i64, vp, i32, vp, i32, i64, i64, i64, f32, vp,
                                                  i64, vp, vp, sz, vp]
        lib.emu_add_rms_norm_backward_workspace.argtypes = [i64, i64]
        lib.emu_add_rms_norm_backward_workspace.restype = sz
        lib.emu_int8_scaled_mm.argtypes = [vp, i64, vp, i64, i64, i64, i64, vp, i32, vp, i32, vp, i32, vp, i32, i64, vp,
                                           sz, vp]
        lib.emu_int8_scaled_mm_workspace.argtypes = [i64, i64, i64, i32]
        lib.emu_int8_scaled_mm_workspace.restype = sz
        lib.emu_token_logprobs.argtypes = [vp, i32, i64, i64, i64, vp, i64, i64, vp, vp, vp, vp, vp, vp, sz, vp]
        lib.emu_token_logprobs_workspace.argtypes = [i64, i64, i64]
        lib.emu_token_logprobs_workspace.restype = sz
        lib.emu_token_logprobs_backward.argtypes = [vp, i32, i64, i64, i64, vp, i64, vp, vp, vp, vp, vp, vp, i64, vp,
                                                    i64, vp]
        _LIB = lib
    return _LIB


def _launch(device, function, *args):
    """function(*args, stream) on torch's current stream of `device`."""
    index = device.index
    if index == torch.cuda.current_device():
        _check(function(*args, torch._C._cuda_getCurrentRawStream(index)))
    else:
        with torch.cuda.device(device):
            _check(function(*args, torch._C._cuda_getCurrentRawStream(index)))


def _workspace(nbytes: int, device):
    return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None


def _ptr(t):
    return None if t is None else t.data_ptr()


def _no_grad(*tensors):
    if torch.is_grad_enabled():
        for t in tensors:
            if t is not None and t.requires_grad:
                raise RuntimeError("an input requires a gradient: call under torch.no_grad() and make the backward call")


def _gpu(name: str, t: torch.Tensor):
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.device


def _float(name: str, t: torch.Tensor, beside=None):
    if t.dtype not in FLOAT_DTYPES or (beside is not None and t.dtype not in (beside, torch.float32)):
        want = "bfloat16, float16 or float32" if beside is None else f"{beside} or float32"
        raise TypeError(f"{name} must be {want}, not {t.dtype}")


def _rows(name: str, t: torch.Tensor):
    """(rows, columns, leading dimension) of a tensor whose leading axes are rows."""
    if t.dim() != 2:
        if t.dim() == 0:
            raise ValueError(f"{name} must have at least one axis")
        try:
            t = t.view(math.prod(t.shape[:-1]), t.shape[-1])
        except RuntimeError:
            raise ValueError(f"{name}'s leading axes must be one axis of rows with one stride") from None
    T, n = t.shape
    if n > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have unit stride along its last axis")
    return T, n, t.stride(0) if T > 1 and n > 0 else n


def _same(name: str, t: torch.Tensor, like: torch.Tensor):
    """The leading dimension of `t`, which has to have the shape and device of `like`."""
    if t.shape != like.shape:
        raise ValueError(f"{name} must have shape {tuple(like.shape)}, not {tuple(t.shape)}")
    _on_device(name, t, like.device)
    return _rows(name, t)[2]


def _vector(name: str, t: torch.Tensor, n: int, device):
    if t.dim() != 1 or t.shape[0] != n or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be a dense vector of {n} values")
    _on_device(name, t, device)


def add_rms_norm_quant(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None, eps: float = 1e-6,
                       out_dtype=torch.float8_e4m3fn, scale: torch.Tensor | None = None,
                       h_out: torch.Tensor | None = None):
    """(codes, scale, h) of ``h = x + residual`` and ``y = h / sqrt(mean(h^2) + eps) * weight``
    along the last axis; ``codes * scale`` stands for y.

    codes: ``out_dtype`` (float8_e4m3fn, float8_e5m2 or int8), y / scale cut to
    the type's largest value and rounded to nearest even.  scale: the
    one-element float32 tensor given (as ``scaled_mm`` takes it), or, where
    none is, one for each row: max(max|y| / largest, 2^-126), shape
    ``[..., 1]`` (as ``int8_scaled_mm`` takes it).  h: of the residual's type
    (x's, or float32), the norm being taken before that rounding; None without
    a residual.  h_out: where to write it, which may be the residual itself.
    A row with a NaN or an infinity in h has the scale NaN."""
    dev = _gpu("x", x)
    _no_grad(x, weight, residual)
    _float("x", x)
    _float("weight", weight, x.dtype)
    T, n, ldx = _rows("x", x)
    _vector("weight", weight, n, dev)
    if out_dtype not in QUANT_DTYPES:
        raise EmuError(EMU_ERR_UNSUPPORTED, f"output dtype {out_dtype} is not supported")
    ldr = ldh = 0
    rdt = 0
    if residual is not None:
        _float("residual", residual, x.dtype)
        rdt = DTYPE[residual.dtype]
        ldr = _same("residual", residual, x)
        if h_out is None:
            h_out = torch.empty(x.shape, dtype=residual.dtype, device=dev)
            ldh = n
        else:
            if h_out.dtype != residual.dtype:
                raise TypeError("h_out must be of the residual's type")
            ldh = _same("h_out", h_out, x)
    elif h_out is not None:
        raise ValueError("h_out needs a residual")
    codes = torch.empty(x.shape, dtype=out_dtype, device=dev)
    own = None
    if scale is None:
        own = torch.empty(x.shape[:-1] + (1,), dtype=torch.float32, device=dev)
    elif scale.numel() != 1 or scale.dtype != torch.float32:
        raise ValueError("scale must be a one-element float32 tensor")
    else:
        _on_device("scale", scale, dev)
    _launch(dev, _lib().emu_add_rms_norm_quant, x.data_ptr(), DTYPE[x.dtype], ldx, weight.data_ptr(),
            DTYPE[weight.dtype], _ptr(residual), rdt, ldr, T, n, eps, codes.data_ptr(), DTYPE[out_dtype], n,
            _ptr(scale), _ptr(own), _ptr(h_out), ldh)
    return codes, scale if own is None else own, h_out


def add_rms_norm_backward(g: torch.Tensor, h: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
                          grad_h: torch.Tensor | None = None):
    """(grad_in, grad_weight) of ``add_rms_norm_quant``, the rounding to 8 bits passed straight through.

    g: the gradient of y (``codes * scale``); h: what the forward call
    returned as h (x where there was no residual); grad_h: the gradient that
    reaches h by itself, along the residual stream.  grad_in, of g's type, is
    the gradient of x and of the residual alike."""
    dev = _gpu("g", g)
    _no_grad(g, h, weight, grad_h)
    _float("g", g)
    _float("h", h, g.dtype)
    _float("weight", weight, g.dtype)
    T, n, ldg = _rows("g", g)
    ldh = _same("h", h, g)
    _vector("weight", weight, n, dev)
    ldgh = ghdt = 0
    if grad_h is not None:
        _float("grad_h", grad_h, g.dtype)
        ghdt = DTYPE[grad_h.dtype]
        ldgh = _same("grad_h", grad_h, g)
    grad_in = torch.empty(g.shape, dtype=g.dtype, device=dev)
    grad_weight = torch.empty(n, dtype=weight.dtype, device=dev)
    lib = _lib()
    nbytes = lib.emu_add_rms_norm_backward_workspace(T, n)
    ws = _workspace(nbytes, dev)
    _launch(dev, lib.emu_add_rms_norm_backward, g.data_ptr(), DTYPE[g.dtype], ldg, h.data_ptr(), DTYPE[h.dtype], ldh,
            weight.data_ptr(), DTYPE[weight.dtype], _ptr(grad_h), ghdt, ldgh, T, n, eps, grad_in.data_ptr(), n,
            grad_weight.data_ptr(), _ptr(ws), nbytes)
    return grad_in, grad_weight


def _mm_scale(name: str, s: torch.Tensor, rows: int, shapes, device) -> int:
    """1 where `s` has a scale for each row, 0 where it has one for all."""
    if not isinstance(s, torch.Tensor) or s.dtype != torch.float32:
        raise ValueError(f"{name} must be a float32 tensor")
    _on_device(name, s, device)
    if s.numel() == 1:
        return 0
    if tuple(s.shape) not in shapes or not s.is_contiguous():
        raise ValueError(f"{name} must be dense with one value, or of shape {' or '.join(map(str, shapes))}")
    return 1


def int8_scaled_mm(mat1: torch.Tensor, mat2: torch.Tensor, scale_a: torch.Tensor, scale_b: torch.Tensor,
                   bias: torch.Tensor | None = None, out_dtype=torch.bfloat16,
                   out: torch.Tensor | None = None) -> torch.Tensor:
    """``(mat1 @ mat2) * scale_a * scale_b + bias`` of int8 operands, the products' sum exact.

    mat1 [M, K] row-major, mat2 [K, N] column-major (``w.t()`` for a row-major
    ``w [N, K]``), as ``scaled_mm`` takes them, but of any sizes up to
    K = 131071 and with no alignment.  scale_a: float32, one value or one for
    each row of mat1 ([M] or [M, 1]); scale_b: one value or one for each column
    of mat2 ([N] or [1, N]).  bias [N] of out_dtype or float32."""
    if mat1.dtype != torch.int8 or mat2.dtype != torch.int8:
        raise TypeError(f"expected int8 operands, got {mat1.dtype} and {mat2.dtype}")
    a, w, M, N, K, lda, ldw = _operands(mat1, mat2)
    dev = a.device
    if out_dtype not in FLOAT_DTYPES:
        raise EmuError(EMU_ERR_UNSUPPORTED, f"output dtype {out_dtype} is not supported")
    per_a = _mm_scale("scale_a", scale_a, M, ((M,), (M, 1)), dev)
    per_b = _mm_scale("scale_b", scale_b, N, ((N,), (1, N)), dev)
    _no_grad(scale_a, scale_b, bias)
    bdt = 0
    if bias is not None:
        _float("bias", bias, out_dtype)
        _vector("bias", bias, N, dev)
        bdt = DTYPE[bias.dtype]
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=dev)
        ldo = N
    else:
        _on_device("out", out, dev)
        if out.shape != (M, N) or out.dtype != out_dtype or (N > 1 and out.stride(1) != 1):
            raise ValueError("out must be a row-major [M, N] tensor of out_dtype")
        ldo = out.stride(0) if M > 1 else N
    lib = _lib()
    ap, wp = a.data_ptr(), w.data_ptr()
    aligned = not (ap | wp | lda | ldw) & 15 and lda <= INT8_MAX_ALIGNED_LD and ldw <= INT8_MAX_ALIGNED_LD
    nbytes = lib.emu_int8_scaled_mm_workspace(M, N, K, aligned)
    ws = _workspace(nbytes, dev)
    _launch(dev, lib.emu_int8_scaled_mm, ap, lda, wp, ldw, M, N, K, scale_a.data_ptr(), per_a, scale_b.data_ptr(),
            per_b, _ptr(bias), bdt, out.data_ptr(), DTYPE[out_dtype], ldo, _ptr(ws), nbytes)
    return out


class TokenLogprobs(NamedTuple):
    """What ``token_logprobs`` returns; the last two are None without alternatives."""
    logprobs: torch.Tensor
    entropy: torch.Tensor
    lse: torch.Tensor
    top_logprobs: torch.Tensor | None
    top_tokens: torch.Tensor | None


def _tokens(tokens: torch.Tensor, logits: torch.Tensor):
    """(dense tokens, C) for tokens of the logits' leading axes, with or without one of their own."""
    lead = logits.shape[:-1]
    if tokens.dtype != torch.int64:
        raise TypeError(f"tokens must be int64, not {tokens.dtype}")
    if tokens.shape != lead and tokens.shape[:-1] != lead:
        raise ValueError(f"tokens must have shape {tuple(lead)}, or that and one axis more, not {tuple(tokens.shape)}")
    _on_device("tokens", tokens, logits.device)
    return tokens.contiguous(), 1 if tokens.shape == lead else tokens.shape[-1]


def _small(name: str, t: torch.Tensor, shape, device, dtype=torch.float32):
    """A dense tensor of one value a row (or few): an expanded gradient is laid out."""
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype:
        raise ValueError(f"{name} must be a {dtype} tensor of shape {tuple(shape)}")
    _on_device(name, t, device)
    return t.contiguous()


def token_logprobs(logits: torch.Tensor, tokens: torch.Tensor, top_k: int = 0) -> TokenLogprobs:
    """Log probabilities of ``tokens`` under softmax(logits) along the last axis, with the
    distribution's entropy, the log of its sum (lse) and its ``top_k`` most likely tokens.

    logits [..., V]; tokens int64 [...] or [..., C], a token below 0 standing
    for none (its log probability is 0).  All outputs are float32, in the
    natural logarithm; top_tokens int64, in falling order, equal logits by
    rising token; top_k <= min(V, 64).  Logits of -inf have probability 0; a
    row of nothing else has lse and log probabilities -inf and entropy 0."""
    dev = _gpu("logits", logits)
    _no_grad(logits)
    _float("logits", logits)
    T, V, ldz = _rows("logits", logits)
    tok, C = _tokens(tokens, logits)
    lead = logits.shape[:-1]
    lp = torch.empty(tok.shape, dtype=torch.float32, device=dev)
    stats = torch.empty((2,) + lead, dtype=torch.float32, device=dev)
    entropy, lse = stats[0], stats[1]
    top_lp = top_tok = None
    if top_k:
        top_lp = torch.empty(lead + (top_k,), dtype=torch.float32, device=dev)
        top_tok = torch.empty(lead + (top_k,), dtype=torch.int64, device=dev)
    lib = _lib()
    nbytes = lib.emu_token_logprobs_workspace(T, V, top_k)
    ws = _workspace(nbytes, dev)
    _launch(dev, lib.emu_token_logprobs, logits.data_ptr(), DTYPE[logits.dtype], ldz, T, V, tok.data_ptr(), C, top_k,
            lp.data_ptr(), entropy.data_ptr(), lse.data_ptr(), _ptr(top_lp), _ptr(top_tok), _ptr(ws), nbytes)
    return TokenLogprobs(lp, entropy, lse, top_lp, top_tok)


def token_logprobs_backward(logits: torch.Tensor, tokens: torch.Tensor, lse: torch.Tensor,
                            entropy: torch.Tensor | None, grad_logprobs: torch.Tensor | None = None,
                            grad_entropy: torch.Tensor | None = None, top_tokens: torch.Tensor | None = None,
                            grad_top: torch.Tensor | None = None, out: torch.Tensor | None = None) -> torch.Tensor:
    """The gradient with respect to the logits, of the logits' type, from those of
    ``token_logprobs``'s outputs (each may be None).

    lse and entropy are the forward call's, and so is top_tokens where
    grad_top is given; entropy may be None where grad_entropy is.  out: where
    to write it, which may be the logits themselves."""
    dev = _gpu("logits", logits)
    _no_grad(logits, lse, entropy, grad_logprobs, grad_entropy, grad_top)
    _float("logits", logits)
    T, V, ldz = _rows("logits", logits)
    tok, C = _tokens(tokens, logits)
    lead = logits.shape[:-1]
    lse = _small("lse", lse, lead, dev)
    if entropy is not None:
        entropy = _small("entropy", entropy, lead, dev)
    if grad_logprobs is not None:
        grad_logprobs = _small("grad_logprobs", grad_logprobs, tok.shape, dev)
    if grad_entropy is not None:
        if entropy is None:
            raise ValueError("grad_entropy needs the entropy")
        grad_entropy = _small("grad_entropy", grad_entropy, lead, dev)
    k = 0
    if grad_top is not None:
        if top_tokens is None:
            raise ValueError("grad_top needs top_tokens")
        k = grad_top.shape[-1] if grad_top.dim() else 0
        grad_top = _small("grad_top", grad_top, lead + (k,), dev)
        top_tokens = _small("top_tokens", top_tokens, lead + (k,), dev, torch.int64)
    if out is None:
        out = torch.empty(logits.shape, dtype=logits.dtype, device=dev)
        ldo = V
    else:
        if out.dtype != logits.dtype:
            raise TypeError("out must be of the logits' type")
        ldo = _same("out", out, logits)
    _launch(dev, _lib().emu_token_logprobs_backward, logits.data_ptr(), DTYPE[logits.dtype], ldz, T, V, tok.data_ptr(),
            C, lse.data_ptr(), _ptr(entropy), _ptr(grad_logprobs), _ptr(grad_entropy), _ptr(top_tokens),
            _ptr(grad_top), k, out.data_ptr(), ldo)
    return out
