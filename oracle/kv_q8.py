"""CPU oracle of the 8-bit paged cache's operators, in float64, one request and
head at a time, from their definitions.

TEST INFRASTRUCTURE: only tests/ (and smoke()) use this module; it shares no
code with the CUDA library.

A cache is a dict of codes k, v (uint8 e4m3 codes [pages, H, P, D]) and scales
ks, vs ([pages, H]); a code stands for code * scale. Position p of request b is
slot p % P of page table[b][p // P].
"""

from __future__ import annotations

import numpy as np

E4M3_MAX = 448.0
STATUS_BAD_PARENT = 2
STATUS_BAD_PAGE = 256


def _table():
    v = np.empty(256)
    for c in range(256):
        e, m = c >> 3 & 15, c & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v[c] = np.nan if c & 127 == 127 else (-x if c & 128 else x)
    return v


VALUES = _table()


def decode(codes):
    return VALUES[np.asarray(codes)]


def encode(x):
    """Nearest e4m3 code, ties to an even code; saturating, NaN to 0x7f."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.where(np.isnan(x), 0.0, np.abs(x)), E4M3_MAX)
    pos = VALUES[:127]
    hi = np.clip(np.searchsorted(pos, a), 1, 126)
    lo = hi - 1
    dl, dh = a - pos[lo], pos[hi] - a
    c = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    c = np.where(a == 0, 0, c) | np.where(np.signbit(x) & ~np.isnan(x), 128, 0)
    return np.where(np.isnan(x), 0x7f, c).astype(np.uint8)


def need_scale(x):
    x = np.abs(np.asarray(x, dtype=np.float64))
    x = x[np.isfinite(x)]
    m = x.max() if x.size else 0.0
    if m == 0:
        return 2.0 ** -100
    e = np.floor(np.log2(m / E4M3_MAX)) - 2
    while m > E4M3_MAX * 2.0 ** e:
        e += 1
    return 2.0 ** min(max(e, -100), 119)


def _page(table, b, lp, pages):
    if lp >= table.shape[1]:
        return -1
    p = int(table[b, lp])
    return p if 0 <= p < pages else -1


def append(cache, k_new, v_new, table, base, path=None, num_acc=None):
    """A copy of the cache after the append, out_len and status."""
    c = {n: a.copy() for n, a in cache.items()}
    pages, H, P, D = c["k"].shape
    B, N = k_new.shape[:2]
    out_len, status = np.array(base, dtype=np.int64), np.zeros(B, dtype=np.int64)
    for b in range(B):
        s, count = int(base[b]), N if num_acc is None else int(num_acc[b]) + 1
        limit = N if path is None else min(N, path.shape[1])
        bad = s < 0 or count < 0 or count > limit or s + count > table.shape[1] * P
        nodes = range(max(count, 0)) if path is None or bad else [int(x) for x in path[b, :count]]
        if not bad:
            bad = any(not 0 <= n < N for n in nodes) or \
                any(_page(table, b, p // P, pages) < 0 for p in range(s, s + count))
        if bad:
            status[b] = STATUS_BAD_PAGE
            continue
        out_len[b] = s + count
        for lp in sorted({p // P for p in range(s, s + count)}):
            page, lo, hi = int(table[b, lp]), max(s, lp * P), min(s + count, (lp + 1) * P)
            for codes, scales, new in ((c["k"], c["ks"], k_new), (c["v"], c["vs"], v_new)):
                for h in range(H):
                    x = np.stack([new[b, nodes[p - s], h] for p in range(lo, hi)])
                    sc, kept = need_scale(x), lo - lp * P
                    if kept:
                        old = scales[page, h]
                        sc = max(sc, old)
                        if sc != old:
                            codes[page, h, :kept] = encode(decode(codes[page, h, :kept]) * (old / sc))
                    codes[page, h, kept:kept + hi - lo] = encode(x / sc)
                    scales[page, h] = sc
    return c, out_len, status


def _dense(cache, which, table, b, h, n):
    """Values [n, D] and which positions have a page."""
    codes, scales = (cache["k"], cache["ks"]) if which == "k" else (cache["v"], cache["vs"])
    pages, _, P, D = codes.shape
    x, there = np.zeros((n, D)), np.zeros(n, dtype=bool)
    for p0 in range(0, n, P):
        page, m = _page(table, b, p0 // P, pages), min(P, n - p0)
        if page >= 0:
            x[p0:p0 + m] = decode(codes[page, h, :m]) * float(scales[page, h])
            there[p0:p0 + m] = True
    return x, there


def _sees(base, n, N, parents):
    """[N, base + n]: which positions each node sees; rows past n see nothing."""
    see = np.zeros((N, base + n), dtype=bool)
    for i in range(min(n, N)):
        see[i, :base] = True
        a = i
        while a >= 0:
            see[i, base + a] = True
            up = a - 1 if parents is None else int(parents[a])
            a = up if up < a else -1
    return see


def attention(q, cache, table, base, parents=None, n_nodes=None, sm=1.0):
    """out, lse, and the bounds sum p |v| and max sum |q||k| sm that errors are measured by."""
    B, N, Hq, D = q.shape
    H = cache["k"].shape[1]
    G = Hq // H
    out, lse = np.zeros((B, N, Hq, D)), np.full((B, N, Hq), -np.inf)
    absv, smax = np.zeros((B, N, Hq, D)), np.zeros((B, N, Hq))
    for b in range(B):
        n = N if n_nodes is None else int(n_nodes[b])
        s = int(base[b])
        see = _sees(s, n, N, None if parents is None else parents[b])
        for h in range(Hq):
            k, there = _dense(cache, "k", table, b, h // G, s + n)
            v, _ = _dense(cache, "v", table, b, h // G, s + n)
            for i in range(N):
                on = see[i] & there
                if not on.any():
                    continue
                kk, vv = k[on], v[on]
                x = kk @ q[b, i, h] * sm
                with np.errstate(invalid="ignore"):
                    m = x.max()
                    p = np.exp(x - m)
                lse[b, i, h] = m + np.log(p.sum())
                p = p / p.sum()
                out[b, i, h] = p @ vv
                absv[b, i, h] = p @ np.abs(vv)
                smax[b, i, h] = (np.abs(kk) @ np.abs(q[b, i, h])).max() * abs(sm)
    return out, lse, absv, smax


def weights(q, lse, cache, table, base, scores, path=None, num_acc=None, sm=1.0, decay=1.0):
    """out_scores, and per entry the bound sum of w (1 + max sum |q||k| sm)."""
    B, N, Hq, D = q.shape
    H, S = scores.shape[1:]
    G = Hq // H
    out, err = np.zeros((B, H, S)), np.zeros((B, H, S))
    for b in range(B):
        s, n = int(base[b]), N if num_acc is None else int(num_acc[b]) + 1
        for h in range(H):
            out[b, h, :s] = decay * scores[b, h, :s]
            k, there = _dense(cache, "k", table, b, h, s + n)
            for i in range(n):
                node = i if path is None else int(path[b, i])
                for g in range(G):
                    hq = h * G + g
                    x = k[:s + i + 1] @ q[b, node, hq] * sm
                    big = np.abs(k[:s + i + 1]) @ np.abs(q[b, node, hq]) * abs(sm)
                    w = np.where(there[:s + i + 1], np.exp(x - lse[b, node, hq]), 0.0)
                    out[b, h, :s + i + 1] += w
                    err[b, h, :s + i + 1] += w * (1 + big + abs(lse[b, node, hq]))
    return out, err


def evict(cache, table, seq_len, scores, positions, keep, sinks=0, protect_from=None):
    """A copy of the cache after eviction, scores, positions, lengths, status."""
    c = {n: a.copy() for n, a in cache.items()}
    pages, H, P, D = c["k"].shape
    B, _, S = scores.shape
    osc, opos = np.zeros_like(scores), np.full_like(positions, -1)
    out_len, status = np.array(seq_len, dtype=np.int64), np.zeros(B, dtype=np.int64)
    for b in range(B):
        n = int(seq_len[b])
        bad = n < 0 or n > S or n > table.shape[1] * P or any(_page(table, b, j, pages) < 0 for j in range(-(-n // P)))
        if bad:
            status[b] = STATUS_BAD_PAGE
        if bad or n <= keep:
            m = min(max(n, 0), S)
            osc[b, :, :m], opos[b, :, :m] = scores[b, :, :m], positions[b, :, :m]
            continue
        out_len[b] = keep
        for h in range(H):
            def rank(j):
                pos, s = positions[b, h, j], float(scores[b, h, j])
                safe = pos < sinks or (protect_from is not None and pos >= protect_from[b])
                return (0, 0.0, j) if safe else (1, np.inf if np.isnan(s) else -s, np.isnan(s), j)
            order = sorted(range(n), key=lambda j: (rank(j)[0], rank(j)[1], rank(j)[-2] if rank(j)[0] else 0, j))
            kept = set(order[:keep])
            src = list(range(keep))
            for to, fr in zip([j for j in range(keep) if j not in kept], [j for j in range(keep, n) if j in kept]):
                src[to] = fr
            osc[b, h, :keep], opos[b, h, :keep] = scores[b, h, src], positions[b, h, src]
            for codes, scales, old_codes, old_scales in ((c["k"], c["ks"], cache["k"], cache["ks"]),
                                                         (c["v"], c["vs"], cache["v"], cache["vs"])):
                for lp in range(keep // P):
                    part = src[lp * P:(lp + 1) * P]
                    at = [int(table[b, j // P]) for j in part]
                    if part == list(range(lp * P, (lp + 1) * P)):
                        continue
                    sc = max(old_scales[a, h] for a in at)
                    page = int(table[b, lp])
                    for i, (j, a) in enumerate(zip(part, at)):
                        if old_scales[a, h] == sc:
                            codes[page, h, i] = old_codes[a, h, j % P]
                        else:
                            codes[page, h, i] = encode(decode(old_codes[a, h, j % P]) * (float(old_scales[a, h]) / float(sc)))
                    scales[page, h] = sc
    return c, osc, opos, out_len, status
