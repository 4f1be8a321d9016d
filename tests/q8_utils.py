"""Inputs of the 8-bit cache's GPU tests: caches with shuffled pages, on the host for the oracle and on the GPU."""

import numpy as np
import torch

import speculative_decoding_verification_72_gb300 as sv
from oracle import kv_q8 as K

DEV = torch.device("cuda:0")


def host_cache(rng, pages, H, P, D, pow2=True):
    """Codes of N(0, 1) rows under scales near 2^-7 (or scales of no special form)."""
    def codes():
        c = K.encode(np.clip(rng.standard_normal((pages, H, P, D)) * 100, -448, 448))
        return c

    def scales():
        s = 2.0 ** rng.integers(-8, -5, (pages, H))
        return (s if pow2 else s * rng.uniform(0.6, 1.7, (pages, H))).astype(np.float32).astype(np.float64)
    return dict(k=codes(), v=codes(), ks=scales(), vs=scales())


def table(rng, lens, P, pages, width=None):
    """Shuffled page ids, -1 where a request has no page."""
    need = [-(-n // P) for n in lens]
    W = max([1, *need]) if width is None else width
    ids = rng.permutation(pages)[:sum(need)]
    t, at = np.full((len(lens), W), -1), 0
    for b, n in enumerate(need):
        t[b, :n] = ids[at:at + n]
        at += n
    return t


def to_gpu(c):
    f8 = lambda a: torch.from_numpy(a.copy()).to(DEV).view(torch.float8_e4m3fn)  # noqa: E731
    f32 = lambda a: torch.from_numpy(a.astype(np.float32)).to(DEV)  # noqa: E731
    return sv.Q8Cache(f8(c["k"]), f8(c["v"]), f32(c["ks"]), f32(c["vs"]))


def to_host(cache):
    u8 = lambda t: t.view(torch.uint8).cpu().numpy()  # noqa: E731
    return dict(k=u8(cache.k), v=u8(cache.v), ks=cache.k_scale.double().cpu().numpy(),
                vs=cache.v_scale.double().cpu().numpy())


def same_cache(got, want):
    for n in ("k", "v", "ks", "vs"):
        assert np.array_equal(got[n], want[n], equal_nan=n in ("ks", "vs")), n


def i32(a):
    return torch.as_tensor(np.asarray(a), dtype=torch.int32, device=DEV)


def rows(rng, shape, dtype, std=1.0):
    x = torch.from_numpy(rng.standard_normal(shape) * std).to(dtype)
    return x.to(DEV), x.double().numpy()


def check_attention(r, want, dtype):
    """out within the rounding of the output type and of P (f16) against sum p |v|; lse within fp32 sums of the scores.

    Scores are sums of D <= 128 exact products in fp32 (error <= 2^-17 of sum |q||k|, and e^x turns that into the same
    relative error of p); P is rounded to 11 bits and the output to 11 (f16) or 8 (bf16)."""
    out, lse, absv, smax = want
    u = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -11
    got, glse = r["out"].double().cpu().numpy(), r["lse"].double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(out))
    assert np.array_equal(np.isinf(glse), np.isinf(lse)) and np.array_equal(np.isnan(glse), np.isnan(lse))
    ok = np.isnan(out) | (np.abs(got - out) <= u * np.abs(out) * 1.01 + (2.0 ** -10 + 2.0 ** -16 * (1 + smax[..., None])) * absv
                          + 2.0 ** -24)
    assert ok.all(), np.abs(got - out)[~ok].max()
    fine = np.isfinite(lse)
    assert (np.abs(glse - lse)[fine] <= 2.0 ** -17 * (1 + smax[fine]) + 2.0 ** -22 * np.abs(lse[fine])).all()
