"""Inputs and tolerances of the 16-bit paged cache's GPU tests."""

import numpy as np
import torch

import speculative_decoding_verification_72_gb300 as sv

DEV = torch.device("cuda:0")
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}   # half a step of the type, relative


def normal(rng, shape, dtype, std=1.0):
    """N(0, std^2) in `dtype`, on the host in 64 bits and on the GPU."""
    x = torch.from_numpy(rng.standard_normal(shape) * std).to(dtype)
    return x.double().numpy(), x.to(DEV)


def host_cache(rng, pages, P, H, D, dtype):
    return dict(k=normal(rng, (pages, P, H, D), dtype)[0], v=normal(rng, (pages, P, H, D), dtype)[0])


def to_gpu(c, dtype, layout="nhd"):
    """PagedCache of a host cache: tokens before heads, heads before tokens, or K and V in one tensor."""
    k, v = (torch.from_numpy(c[n]).to(dtype).to(DEV) for n in ("k", "v"))
    if layout == "hnd":
        k, v = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (k, v))
    elif layout == "joint":
        k, v = torch.stack([k, v], 1).unbind(1)
    return sv.PagedCache(k, v)


def to_host(cache):
    return dict(k=cache.k.double().cpu().numpy(), v=cache.v.double().cpu().numpy())


def table(rng, lens, P, pages, width=None):
    """Shuffled page ids, -1 where a request has no page."""
    need = [-(-max(n, 0) // P) for n in lens]
    W = max([1, *need]) if width is None else width
    ids = rng.permutation(pages)[:sum(need)]
    t, at = np.full((len(lens), W), -1), 0
    for b, n in enumerate(need):
        t[b, :n] = ids[at:at + n]
        at += n
    return t


def i32(a):
    return torch.as_tensor(np.asarray(a), dtype=torch.int32, device=DEV)


def tree(rng, B, N, depth=5):
    """Parents of random trees; node n's parent is an earlier node of depth below `depth`."""
    out = np.zeros((B, N), int)
    for b in range(B):
        par, deep = [-1], [0]
        for n in range(1, N):
            p = int(rng.choice([m for m in range(n) if deep[m] < depth]))
            par.append(p)
            deep.append(deep[p] + 1)
        out[b] = par
    return out


def inv_freq(rot, base=10000.0):
    return (base ** (-np.arange(rot // 2) * 2.0 / rot)).astype(np.float32)


def check_attention(r, want, dtype, rows_of_head, cap=0.0):
    """Output and lse of spec_attention against the oracle's.

    Scores: dot products of D <= 128 exact products, each of D sums off by at most a step of fp32 (2^-23) of the largest
    sum, so 2^-16 of sum |q||k|; the cap's exponential, quotient and product are off by 2^-22 of the cap each; scaling,
    bias and the running maximum by four roundings (2^-24) of numbers of at most |z| + |lse| + cap. An error E of a score
    is one of E in lse and of 2 E in a weight. The weights themselves are off by 2^-21 from the exponential and by their
    rounding where they multiply v: half a step of the type (more than 32 rows a kv head), or of what a first term left
    (2^-16 of a bf16 weight; of an f16 weight 2^-21, as far as f16's smallest numbers reach: 2^-25 / 2^7 of the largest).
    Products are summed over 16 slots at a time, each sum off by 2^-23. The output is rounded once."""
    out, lse, absv, smax, zmax, count = want
    u = U[dtype]
    got, glse = r["out"].double().cpu().numpy(), r["lse"].double().cpu().numpy()
    assert np.array_equal(np.isinf(glse), np.isinf(lse)) and np.array_equal(np.isnan(glse), np.isnan(lse))
    fine = np.isfinite(lse)
    with np.errstate(all="ignore"):
        err = 2.0 ** -16 * smax + 3 * 2.0 ** -22 * cap + 2.0 ** -22 * (zmax + np.abs(np.where(fine, lse, 0.0)) + cap)
        sums = (count / 16 + 8) * 2.0 ** -23
        off = np.abs(glse - lse)[fine]
        assert (off <= (err + sums + 2.0 ** -22)[fine]).all(), (off - (err + sums)[fine]).max()
        weight = u if rows_of_head > 32 else 2.0 ** -15 if dtype == torch.bfloat16 else 2.0 ** -20
        if dtype == torch.float16:
            weight = weight + count[..., None] * 2.0 ** -32
        bound = u * 1.01 * np.abs(out) + (2 * err[..., None] + weight + sums[..., None] + 2.0 ** -20) * absv * 1.01 + 2.0 ** -24
    assert (got[np.isneginf(lse)] == 0).all()   # a row that sees nothing
    usual = np.isfinite(out)
    assert np.array_equal(np.isfinite(got), usual)
    assert (np.abs(got - out)[usual] <= bound[usual]).all(), np.nanmax((np.abs(got - out) / bound)[usual])
