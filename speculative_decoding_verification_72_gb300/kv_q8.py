"""The 8-bit paged cache of the verify step: spec_kv_append_q8, spec_attention_q8,
spec_attention_weights_q8 and spec_kv_evict_q8 (include/spec_verify.h).

As in ``verify``: torch CUDA tensors in, outputs and workspaces allocated by
the call unless given, work enqueued on the current stream of the cache's
device, SpecVerifyError on anything the call cannot take. With ``out`` (and
``workspace``, where a function has one) given, a call allocates nothing.
Calls can be captured in a CUDA graph (torch.cuda.graph); what they allocate
then, a workspace among it, is the graph's own. The arguments are checked and
marshalled by csrc/binding.cpp; ``_SIGS`` declares the C entry points for
direct use.
"""

from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
from typing import NamedTuple

import torch

from .verify import SpecVerifyError, _SIGS, library_path, load_library

SV_F16 = 2

PAGE_SIZES = (16, 32, 64, 128)
HEAD_DIMS = (64, 128)

_P = ctypes.c_void_p
_I32 = ctypes.c_int32
_I64 = ctypes.c_int64
_SZ = ctypes.c_size_t
_F = ctypes.c_float


class _CacheStruct(ctypes.Structure):
    _fields_ = [("k", _P), ("v", _P), ("k_scale", _P), ("v_scale", _P), ("page_table", _P),
                ("num_pages", _I32), ("Hkv", _I32), ("page_size", _I32), ("D", _I32), ("max_pages", _I32)]


class _RowsStruct(ctypes.Structure):
    _fields_ = [("data", _P), ("stride_b", _I64), ("stride_n", _I64), ("stride_h", _I64)]


_C = ctypes.POINTER(_CacheStruct)
_R = ctypes.POINTER(_RowsStruct)

_SIGS.update({
    "spec_kv_append_q8": (_I32, [_C, _R, _R, _I32, _I32, _I32, _P, _P, _I32, _P, _P, _P, _P]),
    "spec_attention_q8_workspace_size": (_SZ, [_I32, _I32, _I32, _I32, _I32]),
    "spec_attention_q8": (_I32, [_R, _I32, _C, _I32, _I32, _I32, _P, _P, _P, _F, _P, _P, _P, _P, _SZ, _P]),
    "spec_attention_weights_q8": (_I32, [_R, _I32, _P, _C, _I32, _I32, _I32, _P, _P, _I32, _P, _F, _F, _P, _P, _I32,
                                         _P, _P]),
    "spec_kv_evict_q8_workspace_size": (_SZ, [_I32, _I32, _I32]),
    "spec_kv_evict_q8": (_I32, [_C, _I32, _P, _P, _P, _I32, _I32, _I32, _P, _P, _P, _P, _P, _P, _SZ, _P]),
})


class Q8Cache(NamedTuple):
    """One layer's cache: k, v [pages, kv heads, page size, head dim] float8_e4m3fn, contiguous; k_scale, v_scale
    [pages, kv heads] float32. A code stands for code * scale. page size 16, 32, 64 or 128; head dim 64 or 128."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor


def q8_cache(pages, kv_heads, page_size, head_dim, device=None):
    """An empty cache (codes zero, scales one) on `device` (default: the current CUDA device)."""
    if page_size not in PAGE_SIZES or head_dim not in HEAD_DIMS or pages < 1 or kv_heads < 1:
        raise SpecVerifyError(f"page_size must be one of {PAGE_SIZES}, head_dim one of {HEAD_DIMS}")
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    codes = [torch.zeros((pages, kv_heads, page_size, head_dim), dtype=torch.float8_e4m3fn, device=dev) for _ in "kv"]
    scales = [torch.ones((pages, kv_heads), dtype=torch.float32, device=dev) for _ in "kv"]
    return Q8Cache(*codes, *scales)


_BINDING = None


def binding():
    """The compiled binding (built in-tree by __graft_entry__.build()), loaded on first use."""
    global _BINDING
    if _BINDING is None:
        load_library()
        path = os.path.join(os.path.dirname(library_path()), "_binding.so")
        if not os.path.exists(path):
            raise SpecVerifyError(f"the binding is not built at {path}; run __graft_entry__.build() first")
        loader = importlib.machinery.ExtensionFileLoader(f"{__package__}._binding", path)
        mod = importlib.util.module_from_spec(importlib.util.spec_from_loader(loader.name, loader))
        loader.exec_module(mod)
        mod.set_up(SpecVerifyError, torch.as_tensor)
        _BINDING = mod
    return _BINDING


def spec_kv_append_q8(cache, k_new, v_new, page_table, seq_base, path_nodes=None, num_accepted=None, out=None):
    """Write new key / value rows into the cache (modified in place). k_new, v_new [B, N, kv heads, head dim] (fp32,
    bf16 or fp16; any strides that are multiples of 16 bytes); row i of request b becomes position seq_base[b] + i.
    After a verify pass, path_nodes and num_accepted (spec_verify_tree's nodes and num_accepted) write the accepted
    rows again over the pass's nodes (the page that also holds earlier positions keeps the largest scale it had, a rejected
    node's among them). Requests must not share the pages written. Returns dict(out_len [B], status [B]); out["out_len"] is another tensor than
    seq_base and num_accepted."""
    return binding().kv_append(cache, k_new, v_new, page_table, seq_base, path_nodes, num_accepted, out)


def spec_attention_q8(q, cache, page_table, seq_base, parents=None, n_nodes=None, sm_scale=None, workspace=None,
                      out=None):
    """Attention of a verify pass's nodes over the cache. q [B, N, heads, head dim] (bf16 or fp16); node n of request b
    is position seq_base[b] + n (already appended) and sees every earlier position of the request, itself, and its
    ancestors by parents [B, N] (None: a chain). n_nodes [B] shortens requests. sm_scale defaults to head dim^-0.5.
    Returns dict(out [B, N, heads, head dim], lse [B, N, heads], status [B])."""
    return binding().attention(q, cache, page_table, seq_base, parents, n_nodes, sm_scale, workspace, out)


def spec_attention_weights_q8(q, lse, cache, page_table, seq_base, scores, path_nodes=None, num_accepted=None,
                              sm_scale=None, decay=1.0, out=None):
    """Accumulate the attention weight that the accepted rows of a verify pass (path_nodes, num_accepted; None: all N
    rows) gave to each position, per kv head: scores [B, kv heads, S] float32 -> dict(scores, status [B]), decay *
    scores plus the weights. q as in spec_attention_q8, lse its result. out["scores"] may be `scores`."""
    return binding().attention_weights(q, lse, cache, page_table, seq_base, scores, path_nodes, num_accepted, sm_scale,
                                       decay, out)


def spec_kv_evict_q8(cache, page_table, seq_len, scores, positions, keep, sinks=0, protect_from=None, workspace=None,
                     out=None):
    """Evict down to `keep` slots (a multiple of the page size) per request and head by score (the cache is modified in
    place; pages past keep fall free; a request that is evicted from must not share its pages with another). scores [B, kv heads, S] float32, positions [B, kv heads, S] int32 (the token each
    slot holds); tokens at positions below `sinks` or from protect_from[b] on are kept first. Returns dict(scores,
    positions [B, kv heads, S], out_len [B], status [B]); out["scores"] / out["positions"] may be the inputs,
    out["out_len"] not seq_len or protect_from."""
    return binding().kv_evict(cache, page_table, seq_len, scores, positions, keep, sinks, protect_from, workspace, out)
