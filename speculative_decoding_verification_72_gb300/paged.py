"""The 16-bit paged cache of the verify step: spec_kv_append_rope and
spec_attention (include/spec_verify.h).

A verify step on it: spec_kv_append_rope writes the new rows and rotates keys
and queries by position, spec_attention attends over the cache,
spec_verify_tree accepts a path, and spec_kv_compact moves the path's rows
into place (a key is rotated by its depth, which is where it lands). As in
``kv_q8``: torch CUDA tensors in, outputs and workspaces allocated by the call
unless given, work enqueued on the current stream of the cache's device,
SpecVerifyError on anything the call cannot take; calls can be captured in a
CUDA graph. They are for serving: tensors that require a gradient are taken, and
what comes back has none. The arguments are checked and marshalled by csrc/binding.cpp;
``_SIGS`` declares the C entry points for direct use.
"""

from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from .kv_q8 import HEAD_DIMS, PAGE_SIZES, _R, binding
from .verify import SpecVerifyError, _SIGS

_P = ctypes.c_void_p
_I32 = ctypes.c_int32
_I64 = ctypes.c_int64
_SZ = ctypes.c_size_t
_F = ctypes.c_float


class _PagedStruct(ctypes.Structure):
    _fields_ = [("k", _P), ("v", _P), ("k_strides", _I64 * 3), ("v_strides", _I64 * 3), ("page_table", _P),
                ("num_pages", _I32), ("Hkv", _I32), ("page_size", _I32), ("D", _I32), ("max_pages", _I32)]


_C = ctypes.POINTER(_PagedStruct)

_SIGS.update({
    "spec_kv_append_rope": (_I32, [_C, _I32, _R, _R, _R, _I32, _I32, _I32, _P, _P, _P, _P, _I32, _I32, _P, _P, _P, _P]),
    "spec_attention_workspace_size": (_SZ, [_I32, _I32, _I32, _I32, _I32]),
    "spec_attention": (_I32, [_R, _I32, _C, _I32, _I32, _I32, _P, _P, _P, _F, _F, _I32, _P, _P, _P, _P, _P, _SZ, _P]),
})


class PagedCache(NamedTuple):
    """One layer's cache: k, v [pages, page size, kv heads, head dim] bf16 or fp16, with any strides that are multiples
    of 16 bytes (elements of a head contiguous; a permuted view of another order, or halves of one tensor, will do). page
    size 16, 32, 64 or 128; head dim 64 or 128."""
    k: torch.Tensor
    v: torch.Tensor


def paged_cache(pages, kv_heads, page_size, head_dim, dtype=torch.bfloat16, device=None):
    """A cache of zeros on `device` (default: the current CUDA device)."""
    if page_size not in PAGE_SIZES or head_dim not in HEAD_DIMS or pages < 1 or kv_heads < 1:
        raise SpecVerifyError(f"page_size must be one of {PAGE_SIZES}, head_dim one of {HEAD_DIMS}")
    if dtype not in (torch.bfloat16, torch.float16):
        raise SpecVerifyError("dtype must be torch.bfloat16 or torch.float16")
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    return PagedCache(*(torch.zeros((pages, page_size, kv_heads, head_dim), dtype=dtype, device=dev) for _ in "kv"))


def spec_kv_append_rope(cache, k_new, v_new, page_table, seq_base, inv_freq, q=None, parents=None, n_nodes=None,
                        interleaved=False, out=None):
    """Write new key / value rows into the cache (modified in place), keys rotated by position, and rotate queries.
    k_new, v_new [B, N, kv heads, head dim] and q [B, N, heads, head dim] have the cache's type (any strides that are
    multiples of 16 bytes). Row n of request b goes to slot seq_base[b] + n; its position is seq_base[b] + its depth by
    parents [B, N] (at most 1024 rows; None: a chain, position = slot). inv_freq [rotary dims / 2] float32: the pair of dims
    (i, i + rotary dims / 2), or (2 i, 2 i + 1) if interleaved, turns by position * inv_freq[i]. n_nodes [B] shortens
    requests. Requests must not share the pages written. Returns dict(out_len [B], status [B]) and, with q given, q
    (contiguous, 0 in rows past n_nodes; out["q"] may be q where that is contiguous). No other output may be one of the
    inputs (for seq_base and n_nodes as out["out_len"] that is checked)."""
    return binding().kv_append_rope(cache, k_new, v_new, page_table, seq_base, inv_freq, q, parents, n_nodes, interleaved,
                                    out)


def spec_attention(q, cache, page_table, seq_base, parents=None, n_nodes=None, sm_scale=None, softcap=0.0, window=0,
                   slopes=None, workspace=None, out=None):
    """Attention of new rows over the cache. q [B, N, heads, head dim] in the cache's type; row n of request b is slot
    seq_base[b] + n (already appended) and sees every earlier slot of the request, itself, and its ancestors by parents
    [B, N] (at most 1024 rows; None: a chain or a prompt, every earlier row). n_nodes [B] shortens requests. sm_scale
    defaults to head dim^-0.5. softcap > 0 caps scores: softcap * tanh(score / softcap). window > 0 hides what is `window`
    or more positions back. slopes [heads] float32 subtracts slope * distance. Positions are as in spec_kv_append_rope.
    Returns dict(out [B, N, heads, head dim], lse [B, N, heads], status [B])."""
    return binding().paged_attention(q, cache, page_table, seq_base, parents, n_nodes, sm_scale, softcap, window, slopes,
                                     workspace, out)
