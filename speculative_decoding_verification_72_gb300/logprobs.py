"""Token log-probabilities with entropy and top alternatives, and their
gradient: ctypes binding of spec_token_logprobs and
spec_token_logprobs_backward (include/spec_verify.h), and ``token_logprobs``,
the pair as one differentiable torch function."""

from __future__ import annotations

import ctypes

import torch

from .verify import SpecVerifyError, _SIGS, _check, _dtype_code, _f32, _rows_view, _ws, load_library
from .kv_q8 import _ints, _out, _p

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
    lib = load_library()
    x, stride = _rows_view(logits, "logits")
    B, R, V = x.shape
    dev, n_top = x.device, int(n_top)
    if not 0 <= n_top <= MAX_TOP_ALTERNATIVES:
        raise SpecVerifyError(f"n_top must lie in [0, {MAX_TOP_ALTERNATIVES}]")
    tok = _ints(tokens, "tokens", (B, R), dev)
    code = _dtype_code(x)
    f, i = torch.float32, torch.int32
    want = {"logprob": ((B, R), f), "entropy": ((B, R), f), "lse": ((B, R), f), "saved": ((B, R, 4), f), "status": ((B, R), i)}
    if n_top:
        want.update(top_tokens=((B, R, n_top), i), top_logprobs=((B, R, n_top), f))
    out = _out(out, want, dev)
    stream = torch.cuda.current_stream(dev).cuda_stream
    need = lib.spec_token_logprobs_workspace_size(B * R, V, code, n_top)
    if need == 0:
        raise SpecVerifyError("invalid sizes")
    ws = _ws(workspace, need, dev, stream)
    _check(lib.spec_token_logprobs(x.data_ptr(), code, stride, tok.data_ptr(), B * R, V, float(temperature), n_top,
                                   out["logprob"].data_ptr(), out["entropy"].data_ptr(), out["lse"].data_ptr(),
                                   out["saved"].data_ptr(), _p(out["top_tokens"]) if n_top else None,
                                   _p(out["top_logprobs"]) if n_top else None, out["status"].data_ptr(), ws.data_ptr(),
                                   ws.numel() * ws.element_size(), stream))
    return out


def spec_token_logprobs_backward(logits, tokens, saved, grad_logprob, grad_entropy=None, temperature=1.0, out=None):
    """Gradient [B, R, V] (logits' dtype) of sum(grad_logprob * logprob + grad_entropy * entropy); `saved` is
    spec_token_logprobs' for the same logits, tokens and temperature. `out` may be a [B, R, V] tensor, `logits` itself
    among them."""
    lib = load_library()
    x, stride = _rows_view(logits, "logits")
    B, R, V = x.shape
    dev = x.device
    tok = _ints(tokens, "tokens", (B, R), dev)
    if tuple(saved.shape) != (B, R, 4) or saved.dtype != torch.float32 or saved.device != dev or not saved.is_contiguous():
        raise SpecVerifyError(f"saved must be spec_token_logprobs' contiguous float32 {(B, R, 4)} tensor")
    g = _f32(grad_logprob, "grad_logprob", (B, R), dev)
    h = None if grad_entropy is None else _f32(grad_entropy, "grad_entropy", (B, R), dev)
    if out is None:
        out, ostride = torch.empty((B, R, V), dtype=x.dtype, device=dev), V
    else:
        if tuple(out.shape) != (B, R, V) or out.dtype != x.dtype or out.device != dev:
            raise SpecVerifyError(f"out must be a {(B, R, V)} {x.dtype} tensor on {dev}")
        view, ostride = _rows_view(out, "out")
        if view is not out:
            raise SpecVerifyError("out must have evenly strided rows of unit stride")
    _check(lib.spec_token_logprobs_backward(x.data_ptr(), _dtype_code(x), stride, tok.data_ptr(), saved.data_ptr(),
                                            g.data_ptr(), _p(h), B * R, V, float(temperature), out.data_ptr(), ostride,
                                            torch.cuda.current_stream(dev).cuda_stream))
    return out


class _TokenLogprobs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, tokens, temperature):
        r = spec_token_logprobs(logits, tokens, temperature)
        ctx.save_for_backward(logits, tokens, r["saved"])
        ctx.temperature = temperature
        return r["logprob"], r["entropy"]

    @staticmethod
    def backward(ctx, g, h):
        logits, tokens, saved = ctx.saved_tensors
        return spec_token_logprobs_backward(logits, tokens, saved, g, h, ctx.temperature), None, None


def token_logprobs(logits, tokens, temperature=1.0):
    """(logprob, entropy), each [B, R] float32, of spec_token_logprobs; differentiable with respect to logits."""
    return _TokenLogprobs.apply(logits, tokens, temperature)
