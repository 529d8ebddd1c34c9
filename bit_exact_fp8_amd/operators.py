"""The operators beside the FP8 product (C ABI in ``include/emu_operators.h``).

``add_rms_norm_quant`` / ``add_rms_norm_backward``: the residual's addition
with the RMS norm and 8-bit codes, and its gradient.  ``int8_scaled_mm``: the
product of 8-bit integers with scales per token and channel.
``token_logprobs`` / ``token_logprobs_backward``: log probabilities of given
tokens with entropy and top alternatives, and their gradient.

As in ``api``: argument checks and marshalling only (compiled, in
``csrc/ops_binding.cpp``), every step runs in the HIP library's kernels on
torch's current stream of the operands' device, and there is no CPU fallback.
Calls take no part in autograd: the backward calls are the caller's to make,
an input or a given output that requires a gradient is refused while gradients
are enabled, and one with a forward-mode tangent always.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from . import api

MAX_TOP_TOKENS = 64          # EMU_MAX_TOP_TOKENS
MAX_GRAD_TOKENS = 1024       # EMU_MAX_GRAD_TOKENS

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


_OPS = None


def _binding():
    global _OPS
    if _OPS is None:
        _lib()  # (its functions are what the binding calls)
        try:
            from . import _ops
        except ImportError as e:
            raise RuntimeError("the operators' binding _ops.so is not built: run __graft_entry__.build()") from e
        _OPS = _ops
    return _OPS


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
    return (_OPS or _binding()).add_rms_norm_quant(x, weight, residual, eps, out_dtype, scale, h_out)


def add_rms_norm_backward(g: torch.Tensor, h: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
                          grad_h: torch.Tensor | None = None):
    """(grad_in, grad_weight) of ``add_rms_norm_quant``, the rounding to 8 bits passed straight through.

    g: the gradient of y (``codes * scale``); h: what the forward call
    returned as h (x where there was no residual); grad_h: the gradient that
    reaches h by itself, along the residual stream.  grad_in, of g's type, is
    the gradient of x and of the residual alike."""
    return (_OPS or _binding()).add_rms_norm_backward(g, h, weight, eps, grad_h)


def int8_scaled_mm(mat1: torch.Tensor, mat2: torch.Tensor, scale_a: torch.Tensor, scale_b: torch.Tensor,
                   bias: torch.Tensor | None = None, out_dtype=torch.bfloat16,
                   out: torch.Tensor | None = None) -> torch.Tensor:
    """``(mat1 @ mat2) * scale_a * scale_b + bias`` of int8 operands, the products' sum exact.

    mat1 [M, K] row-major, mat2 [K, N] column-major (``w.t()`` for a row-major
    ``w [N, K]``), as ``scaled_mm`` takes them, but of any sizes up to
    K = 131071 and with no alignment.  scale_a: float32, one value or one for
    each row of mat1 ([M] or [M, 1]); scale_b: one value or one for each column
    of mat2 ([N] or [1, N]).  bias [N] of out_dtype or float32."""
    return (_OPS or _binding()).int8_scaled_mm(mat1, mat2, scale_a, scale_b, bias, out_dtype, out)


class TokenLogprobs(NamedTuple):
    """What ``token_logprobs`` returns; the last two are None without alternatives."""
    logprobs: torch.Tensor
    entropy: torch.Tensor
    lse: torch.Tensor
    top_logprobs: torch.Tensor | None
    top_tokens: torch.Tensor | None


def token_logprobs(logits: torch.Tensor, tokens: torch.Tensor, top_k: int = 0) -> TokenLogprobs:
    """Log probabilities of ``tokens`` under softmax(logits) along the last axis, with the
    distribution's entropy, the log of its sum (lse) and its ``top_k`` most likely tokens.

    logits [..., V]; tokens int64 [...] or [..., C], a token below 0 standing
    for none (its log probability is 0).  All outputs are float32, in the
    natural logarithm; top_tokens int64, in falling order, equal logits by
    rising token; top_k <= min(V, MAX_TOP_TOKENS).  Logits of -inf have
    probability 0; a row of nothing else has lse and log probabilities -inf and
    entropy 0.  Any number of tokens a row; the backward call takes
    MAX_GRAD_TOKENS."""
    return TokenLogprobs(*(_OPS or _binding()).token_logprobs(logits, tokens, top_k))


def token_logprobs_backward(logits: torch.Tensor, tokens: torch.Tensor, lse: torch.Tensor,
                            entropy: torch.Tensor | None, grad_logprobs: torch.Tensor | None = None,
                            grad_entropy: torch.Tensor | None = None, top_tokens: torch.Tensor | None = None,
                            grad_top: torch.Tensor | None = None, out: torch.Tensor | None = None) -> torch.Tensor:
    """The gradient with respect to the logits, of the logits' type, from those of
    ``token_logprobs``'s outputs (each may be None).

    lse and entropy are the forward call's, and so is top_tokens where
    grad_top is given; entropy may be None where grad_entropy is.  A row's
    gradients of tokens and of alternatives are at most MAX_GRAD_TOKENS (1024)
    together.  out: where to write it, which may be the logits themselves."""
    return (_OPS or _binding()).token_logprobs_backward(logits, tokens, lse, entropy, grad_logprobs, grad_entropy,
                                                         top_tokens, grad_top, out)
