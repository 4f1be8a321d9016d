"""The 8-bit paged cache of the verify step: ctypes binding of spec_kv_append_q8,
spec_attention_q8, spec_attention_weights_q8 and spec_kv_evict_q8
(include/spec_verify.h).

As in ``verify``: argument marshalling only, torch CUDA tensors in, outputs and
workspaces allocated here unless given, work enqueued on the current stream of
the cache's device, SpecVerifyError on anything the call cannot take. With
``out`` (and ``workspace``, where a function has one) given, a call allocates
nothing and can be captured in a CUDA graph.
"""

from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from .verify import SV_BF16, SV_F32, SpecVerifyError, _SIGS, _check, _ws, load_library

SV_F16 = 2

PAGE_SIZES = (16, 32, 64, 128)
HEAD_DIMS = (64, 128)

_DTYPES = {torch.float32: SV_F32, torch.bfloat16: SV_BF16, torch.float16: SV_F16}

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


def _cache_struct(cache, page_table, B):
    k, v, ks, vs = cache
    if k.dim() != 4 or k.dtype != torch.float8_e4m3fn or not k.is_cuda:
        raise SpecVerifyError("cache.k must be a CUDA float8_e4m3fn tensor [pages, kv heads, page size, head dim]")
    shape, dev = k.shape, k.device
    if v.dtype != k.dtype or v.shape != shape or v.device != dev or not k.is_contiguous() or not v.is_contiguous():
        raise SpecVerifyError("cache.k and cache.v must be contiguous, of one shape and on one device")
    for s in (ks, vs):
        if s.dtype != torch.float32 or s.shape != shape[:2] or s.device != dev or not s.is_contiguous():
            raise SpecVerifyError(f"cache scales must be contiguous float32 {tuple(shape[:2])} tensors on {dev}")
    pages, H, P, D = shape
    if P not in PAGE_SIZES or D not in HEAD_DIMS:
        raise SpecVerifyError(f"page size must be one of {PAGE_SIZES} and head dim one of {HEAD_DIMS}, got {P} and {D}")
    if page_table.dim() != 2:
        raise SpecVerifyError("page_table must be [B, max_pages]")
    page_table = _ints(page_table, "page_table", (B, page_table.shape[1]), dev)
    c = _CacheStruct(k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr(), page_table.data_ptr(), pages, H, P, D,
                     page_table.shape[1])
    return c, page_table, dev, H, P, D


def _ints(t, name, shape, dev):
    """int32 contiguous tensor on dev, the caller's own where it is one."""
    if not isinstance(t, torch.Tensor):
        t = torch.as_tensor(t, dtype=torch.int64)
    if tuple(t.shape) != tuple(shape):
        raise SpecVerifyError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype is torch.int32 and t.device == dev and t.is_contiguous():
        return t
    return t.to(device=dev, dtype=torch.int32).contiguous()


def _rows(t, name, heads, D, dev, dtypes):
    """(struct, tensor) of a [B, N, heads, D] tensor; one that the kernels cannot read as it lies is copied."""
    if t.dim() != 4 or t.shape[2] != heads or t.shape[3] != D or t.device != dev or t.dtype not in dtypes:
        raise SpecVerifyError(f"{name} must be [B, N, {heads}, {D}] of {dtypes} on {dev}, got {tuple(t.shape)} {t.dtype}")
    es = t.element_size()
    sb, sn, sh, sd = t.stride()
    if sd != 1 or t.data_ptr() % 16 or sb * es % 16 or sn * es % 16 or sh * es % 16:
        t = t.contiguous()
        if t.data_ptr() % 16:
            t = t.clone()
        sb, sn, sh, sd = t.stride()
    return _RowsStruct(t.data_ptr(), sb, sn, sh), t


def _path(path_nodes, num_accepted, B, dev):
    if path_nodes is not None and num_accepted is None:
        raise SpecVerifyError("path_nodes needs num_accepted")
    cols = 0
    if path_nodes is not None:
        if path_nodes.dim() != 2:
            raise SpecVerifyError("path_nodes must be [B, columns]")
        cols = path_nodes.shape[1]
        path_nodes = _ints(path_nodes, "path_nodes", (B, cols), dev)
    if num_accepted is not None:
        num_accepted = _ints(num_accepted, "num_accepted", (B,), dev)
    return path_nodes, cols, num_accepted


def _out(out, names, dev):
    """The caller's outputs, checked, or fresh ones: names is {name: (shape, dtype)}."""
    if out is None:
        return {k: torch.empty(shape, dtype=dt, device=dev) for k, (shape, dt) in names.items()}
    for k, (shape, dt) in names.items():
        t = out.get(k)
        if t is None or tuple(t.shape) != tuple(shape) or t.dtype != dt or t.device != dev or not t.is_contiguous():
            raise SpecVerifyError(f"out[{k!r}] must be a contiguous {tuple(shape)} {dt} tensor on {dev}")
    return out


def _p(t):
    return None if t is None else t.data_ptr()


def spec_kv_append_q8(cache, k_new, v_new, page_table, seq_base, path_nodes=None, num_accepted=None, out=None):
    """Write new key / value rows into the cache (modified in place). k_new, v_new [B, N, kv heads, head dim] (fp32,
    bf16 or fp16; any strides that are multiples of 16 bytes); row i of request b becomes position seq_base[b] + i.
    After a verify pass, path_nodes and num_accepted (spec_verify_tree's nodes and num_accepted) write the accepted
    rows again over the pass's nodes. Returns dict(out_len [B], status [B])."""
    lib = load_library()
    B, N = k_new.shape[:2]
    c, table, dev, H, P, D = _cache_struct(cache, page_table, B)
    if k_new.dtype != v_new.dtype or k_new.shape != v_new.shape:
        raise SpecVerifyError("k_new and v_new must have one shape and dtype")
    kr, k_new = _rows(k_new, "k_new", H, D, dev, tuple(_DTYPES))
    vr, v_new = _rows(v_new, "v_new", H, D, dev, tuple(_DTYPES))
    base = _ints(seq_base, "seq_base", (B,), dev)
    path, cols, n_acc = _path(path_nodes, num_accepted, B, dev)
    out = _out(out, {"out_len": ((B,), torch.int32), "status": ((B,), torch.int32)}, dev)
    if N == 0:
        raise SpecVerifyError("k_new must have at least one row per request")
    _check(lib.spec_kv_append_q8(c, kr, vr, _DTYPES[k_new.dtype], B, N, base.data_ptr(), _p(path), cols, _p(n_acc),
                                 out["out_len"].data_ptr(), out["status"].data_ptr(),
                                 torch.cuda.current_stream(dev).cuda_stream))
    return out


def spec_attention_q8(q, cache, page_table, seq_base, parents=None, n_nodes=None, sm_scale=None, workspace=None,
                      out=None):
    """Attention of a verify pass's nodes over the cache. q [B, N, heads, head dim] (bf16 or fp16); node n of request b
    is position seq_base[b] + n (already appended) and sees every earlier position of the request, itself, and its
    ancestors by parents [B, N] (None: a chain). n_nodes [B] shortens requests. sm_scale defaults to head dim^-0.5.
    Returns dict(out [B, N, heads, head dim], lse [B, N, heads], status [B])."""
    lib = load_library()
    B, N, Hq = q.shape[:3]
    c, table, dev, H, P, D = _cache_struct(cache, page_table, B)
    if Hq % H != 0 or Hq == 0:
        raise SpecVerifyError(f"q's heads ({Hq}) must be a multiple of the cache's ({H})")
    qr, q = _rows(q, "q", Hq, D, dev, (torch.bfloat16, torch.float16))
    base = _ints(seq_base, "seq_base", (B,), dev)
    par = None if parents is None else _ints(parents, "parents", (B, N), dev)
    nn = None if n_nodes is None else _ints(n_nodes, "n_nodes", (B,), dev)
    out = _out(out, {"out": ((B, N, Hq, D), q.dtype), "lse": ((B, N, Hq), torch.float32), "status": ((B,), torch.int32)}, dev)
    stream = torch.cuda.current_stream(dev).cuda_stream
    need = lib.spec_attention_q8_workspace_size(B, N, Hq, H, D)
    if need == 0:
        raise SpecVerifyError("invalid sizes")
    ws = _ws(workspace, need, dev, stream)
    _check(lib.spec_attention_q8(qr, _DTYPES[q.dtype], c, B, N, Hq, base.data_ptr(), _p(par), _p(nn),
                                 D ** -0.5 if sm_scale is None else float(sm_scale), out["out"].data_ptr(),
                                 out["lse"].data_ptr(), out["status"].data_ptr(), ws.data_ptr(),
                                 ws.numel() * ws.element_size(), stream))
    return out


def spec_attention_weights_q8(q, lse, cache, page_table, seq_base, scores, path_nodes=None, num_accepted=None,
                              sm_scale=None, decay=1.0, out=None):
    """Accumulate the attention weight that the accepted rows of a verify pass (path_nodes, num_accepted; None: all N
    rows) gave to each position, per kv head: scores [B, kv heads, S] float32 -> dict(scores, status [B]), decay *
    scores plus the weights. q as in spec_attention_q8, lse its result. out["scores"] may be `scores`."""
    lib = load_library()
    B, N, Hq = q.shape[:3]
    c, table, dev, H, P, D = _cache_struct(cache, page_table, B)
    if Hq % H != 0 or Hq == 0:
        raise SpecVerifyError(f"q's heads ({Hq}) must be a multiple of the cache's ({H})")
    qr, q = _rows(q, "q", Hq, D, dev, (torch.bfloat16, torch.float16))
    base = _ints(seq_base, "seq_base", (B,), dev)
    path, cols, n_acc = _path(path_nodes, num_accepted, B, dev)
    S = scores.shape[-1]
    for name, t, shape in (("scores", scores, (B, H, S)), ("lse", lse, (B, N, Hq))):
        if tuple(t.shape) != shape or t.dtype != torch.float32 or t.device != dev or not t.is_contiguous():
            raise SpecVerifyError(f"{name} must be a contiguous float32 {shape} tensor on {dev}")
    out = _out(out, {"scores": ((B, H, S), torch.float32), "status": ((B,), torch.int32)}, dev)
    _check(lib.spec_attention_weights_q8(qr, _DTYPES[q.dtype], lse.data_ptr(), c, B, N, Hq, base.data_ptr(), _p(path),
                                         cols, _p(n_acc), D ** -0.5 if sm_scale is None else float(sm_scale),
                                         float(decay), scores.data_ptr(), out["scores"].data_ptr(), S,
                                         out["status"].data_ptr(), torch.cuda.current_stream(dev).cuda_stream))
    return out


def spec_kv_evict_q8(cache, page_table, seq_len, scores, positions, keep, sinks=0, protect_from=None, workspace=None,
                     out=None):
    """Evict down to `keep` slots (a multiple of the page size) per request and head by score (the cache is modified in
    place; pages past keep fall free). scores [B, kv heads, S] float32, positions [B, kv heads, S] int32 (the token each
    slot holds); tokens at positions below `sinks` or from protect_from[b] on are kept first. Returns dict(scores,
    positions [B, kv heads, S], out_len [B], status [B]); out["scores"] / out["positions"] may be the inputs."""
    lib = load_library()
    B = seq_len.shape[0]
    c, table, dev, H, P, D = _cache_struct(cache, page_table, B)
    S, keep = scores.shape[-1], int(keep)
    for name, t, dt in (("scores", scores, torch.float32), ("positions", positions, torch.int32)):
        if tuple(t.shape) != (B, H, S) or t.dtype != dt or t.device != dev or not t.is_contiguous():
            raise SpecVerifyError(f"{name} must be a contiguous {dt} {(B, H, S)} tensor on {dev}")
    if keep < P or keep % P or keep > S:
        raise SpecVerifyError(f"keep must be a positive multiple of the page size {P}, at most {S}")
    n = _ints(seq_len, "seq_len", (B,), dev)
    pf = None if protect_from is None else _ints(protect_from, "protect_from", (B,), dev)
    out = _out(out, {"scores": ((B, H, S), torch.float32), "positions": ((B, H, S), torch.int32),
                     "out_len": ((B,), torch.int32), "status": ((B,), torch.int32)}, dev)
    stream = torch.cuda.current_stream(dev).cuda_stream
    ws = _ws(workspace, lib.spec_kv_evict_q8_workspace_size(B, H, keep), dev, stream)
    _check(lib.spec_kv_evict_q8(c, B, n.data_ptr(), scores.data_ptr(), positions.data_ptr(), S, keep, int(sinks), _p(pf),
                                out["scores"].data_ptr(), out["positions"].data_ptr(), out["out_len"].data_ptr(),
                                out["status"].data_ptr(), ws.data_ptr(), ws.numel() * ws.element_size(), stream))
    return out
