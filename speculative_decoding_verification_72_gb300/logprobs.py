"""Token log-probabilities with entropy and top alternatives, and their
gradient: spec_token_logprobs and spec_token_logprobs_backward
(include/spec_verify.h), and ``token_logprobs``, the pair as one differentiable
torch function. Arguments are checked and marshalled by csrc/binding.cpp."""

from __future__ import annotations

import ctypes

import torch

from .verify import SpecVerifyError, _SIGS
from .kv_q8 import binding

MAX_TOP_ALTERNATIVES = 32

_V = ctypes.c_void_p
_I32 = ctypes.c_int32
_I64 = ctypes.c_int64
_SZ = ctypes.c_size_t
_F = ctypes.c_float

_SIGS.update({
    "spec_token_logprobs_workspace_size": (_SZ, [_I32, _I32, _I32, _I32]),
    "spec_token_logprobs": (_I32, [_V, _I32, _I64, _V, _I32, _I32, _F, _I32, _V, _V, _V, _V, _V, _V, _V, _V, _SZ, _V]),
    "spec_token_logprobs_backward": (_I32, [_V, _I32, _I64, _V, _V, _V, _V, _I32, _I32, _F, _V, _I64, _V]),
})


def spec_token_logprobs(logits, tokens, temperature=1.0, n_top=0, workspace=None, out=None):
    """Log-probs of given tokens under softmax(logits / temperature). logits [B, R, V] (bf16 / fp32, CUDA), tokens
    [B, R] (-1: no token, log-prob 0). Returns a dict of CUDA tensors: logprob, entropy, lse [B, R], status [B, R],
    saved [B, R, 4] (for the gradient) and, with n_top > 0 (at most 32), top_tokens and top_logprobs [B, R, n_top] in
    descending order, ties to the lower index, -1 and -inf past the last unmasked token."""
    return binding().token_logprobs(logits, tokens, temperature, n_top, workspace, out)


def spec_token_logprobs_backward(logits, tokens, saved, grad_logprob, grad_entropy=None, temperature=1.0, out=None):
    """Gradient [B, R, V] (logits' dtype) of sum(grad_logprob * logprob + grad_entropy * entropy); `saved` is
    spec_token_logprobs' for the same logits, tokens and temperature. `out` may be a [B, R, V] tensor, `logits` itself
    among them."""
    return binding().token_logprobs_backward(logits, tokens, saved, grad_logprob, grad_entropy, temperature, out)


class _TokenLogprobs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, tokens, temperature):
        r = spec_token_logprobs(logits, tokens, temperature)
        ctx.save_for_backward(logits, tokens, r["saved"])
        ctx.temperature = temperature
        return r["logprob"], r["entropy"]

    @staticmethod
    def backward(ctx, g, h):
        return _TokenLogprobsGrad.apply(*ctx.saved_tensors, g, h, ctx.temperature), None, None


class _TokenLogprobsGrad(torch.autograd.Function):
    """The gradient, with an error in place of the second derivative: with create_graph=True the gradient depends on
    logits even where g and h do not require one, and must not count as a constant."""

    @staticmethod
    def forward(ctx, logits, tokens, saved, g, h, temperature):
        return spec_token_logprobs_backward(logits, tokens, saved, g, h, temperature)

    @staticmethod
    def backward(ctx, d):
        raise SpecVerifyError("token_logprobs can be differentiated once, not twice")


def token_logprobs(logits, tokens, temperature=1.0):
    """(logprob, entropy), each [B, R] float32, of spec_token_logprobs; differentiable with respect to logits, once (a
    second derivative raises SpecVerifyError)."""
    return _TokenLogprobs.apply(logits, torch.as_tensor(tokens), temperature)
