"""CPU oracle of token log-probabilities, entropy, top alternatives and their
gradient, in float64, from their definitions.

TEST INFRASTRUCTURE: only tests/ (and smoke()) use this module; it shares no
code with the CUDA library.
"""

from __future__ import annotations

import numpy as np

STATUS_BAD_TOKEN = 1
STATUS_NONFINITE_ROW = 4


def token_logprobs(x, tokens, T=1.0, n_top=0):
    """x [rows, V], tokens [rows] -> dict of logprob, entropy, lse, status [rows], top_tokens, top_logprobs."""
    rows, V = x.shape
    r = dict(logprob=np.zeros(rows), entropy=np.zeros(rows), lse=np.zeros(rows), status=np.zeros(rows, dtype=np.int64),
             top_tokens=np.full((rows, n_top), -1), top_logprobs=np.full((rows, n_top), -np.inf))
    for i in range(rows):
        t, row = int(tokens[i]), x[i].astype(np.float64)
        if t < -1 or t >= V:
            r["status"][i] |= STATUS_BAD_TOKEN
        given = 0 <= t < V
        if np.isnan(row).any() or (row == np.inf).any():
            r["status"][i] |= STATUS_NONFINITE_ROW
            r["entropy"][i] = r["lse"][i] = np.nan
            r["logprob"][i] = np.nan if given else 0.0
            r["top_logprobs"][i] = np.nan
            continue
        on = np.isfinite(row)
        if not on.any():
            r["status"][i] |= STATUS_NONFINITE_ROW
            r["lse"][i] = -np.inf
            r["logprob"][i] = -np.inf if given else 0.0
            continue
        z = row / T
        m = z[on].max()
        lse = m + np.log(np.exp(z[on] - m).sum())
        lp = np.where(on, z - lse, -np.inf)
        p = np.exp(lp)
        r["lse"][i], r["entropy"][i] = lse, -(p[p > 0] * lp[p > 0]).sum()
        r["logprob"][i] = lp[t] if given else 0.0
        order = [j for j in np.argsort(-row, kind="stable") if on[j]][:n_top]
        r["top_tokens"][i, :len(order)], r["top_logprobs"][i, :len(order)] = order, lp[order]
    return r


def backward(x, tokens, g, h, T=1.0):
    """Gradient [rows, V] of sum(g * logprob + h * entropy)."""
    rows, V = x.shape
    d = np.zeros((rows, V))
    r = token_logprobs(x, tokens, T)
    for i in range(rows):
        t = int(tokens[i])
        gi = g[i] if 0 <= t < V else 0.0
        if np.isnan(r["lse"][i]):
            d[i] = np.nan
            continue
        if r["lse"][i] == -np.inf:
            continue
        lp = x[i].astype(np.float64) / T - r["lse"][i]
        p = np.exp(lp)
        d[i] = -gi * p - h[i] * np.where(p > 0, p * (np.where(p > 0, lp, 0.0) + r["entropy"][i]), 0.0)
        if 0 <= t < V:
            d[i, t] += gi
        d[i] /= T
    return d
