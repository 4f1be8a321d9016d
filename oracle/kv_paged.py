"""The 16-bit paged cache in 64 bits: appending with rotation, and attention
with tree masks, caps, windows and biases (include/spec_verify.h). Test
infrastructure; one row at a time, straight from the definitions."""

import numpy as np

STATUS_BAD_PAGE, STATUS_BAD_PARENT = 256, 2


def up(parents, n):
    p = int(parents[n])
    return p if 0 <= p < n else -1


def path(parents, n):
    """Node n and its ancestors, itself first."""
    out = [n]
    while up(parents, out[-1]) >= 0:
        out.append(up(parents, out[-1]))
    return out


def bad_tree(parents, n):
    return any((p != -1) if i == 0 else not 0 <= p < i for i, p in enumerate(parents[:n]))


def depths(parents, N):
    return np.array([len(path(parents, n)) - 1 for n in range(N)]) if parents is not None else np.arange(N)


def turn(x, positions, inv_freq, interleaved=False):
    """Rows x [N, heads, D] turned by angles positions [N] * inv_freq [R / 2]."""
    x = np.array(x, dtype=np.float64)
    half = len(inv_freq)
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    # the fraction of a turn in extended precision: far positions have angles of thousands of turns
    angle = np.asarray(positions, np.longdouble)[:, None, None] * np.asarray(inv_freq, np.float32).astype(np.longdouble)
    c, s = np.cos(angle).astype(np.float64), np.sin(angle).astype(np.float64)
    first, second = x[..., a].copy(), x[..., b].copy()
    x[..., a], x[..., b] = first * c - second * s, second * c + first * s
    return x


def slot(table, b, p, P, pages):
    """(page, row) of slot p of request b, or None."""
    lp = p // P
    if not 0 <= lp < table.shape[1] or not 0 <= table[b, lp] < pages:
        return None
    return int(table[b, lp]), p % P


def append_rope(cache, k_new, v_new, table, base, inv_freq, q=None, parents=None, n_nodes=None, interleaved=False):
    """cache dict(k, v [pages, P, H, D] float64) -> (cache, out_len, status, q)."""
    cache = {n: cache[n].copy() for n in ("k", "v")}
    pages, P = cache["k"].shape[:2]
    B, N = k_new.shape[:2]
    out_len, status = np.array(base, dtype=np.int64), np.zeros(B, int)
    turned = None if q is None else np.zeros(q.shape)
    for b in range(B):
        n = N if n_nodes is None else int(n_nodes[b])
        if not 0 <= n <= N:
            status[b] |= STATUS_BAD_PAGE
            n = min(max(n, 0), N)
        at = int(base[b])
        spots = [slot(table, b, at + i, P, pages) if at >= 0 else None for i in range(n)]
        if at < 0 or None in spots or (n == 0 and at > table.shape[1] * P):
            status[b] |= STATUS_BAD_PAGE
        tree = None if parents is None else parents[b]
        if tree is not None and bad_tree(tree, n):
            status[b] |= STATUS_BAD_PARENT
        pos = at + depths(tree, n)
        if q is not None and at >= 0:
            turned[b, :n] = turn(q[b, :n], pos, inv_freq, interleaved)
        if status[b] & STATUS_BAD_PAGE:
            continue
        rows = turn(k_new[b, :n], pos, inv_freq, interleaved)
        for i, (page, r) in enumerate(spots):
            cache["k"][page, r], cache["v"][page, r] = rows[i], v_new[b, i]
        out_len[b] += n
    return cache, out_len, status, turned


def attention(q, cache, table, base, parents=None, n_nodes=None, sm=1.0, cap=0.0, window=0, slopes=None):
    """(out, lse, sum p |v|, largest sum |q| |k| sm, largest |score|, slots seen) of q [B, N, Hq, D]."""
    pages, P, H, D = cache["k"].shape
    B, N, Hq, _ = q.shape
    G = Hq // H
    out, absv = np.zeros(q.shape), np.zeros(q.shape)
    lse = np.full((B, N, Hq), -np.inf)
    smax, zmax, count = np.zeros((B, N, Hq)), np.zeros((B, N, Hq)), np.zeros((B, N, Hq))
    with np.errstate(all="ignore"):
        for b in range(B):
            at, n = int(base[b]), N if n_nodes is None else min(max(int(n_nodes[b]), 0), N)
            if at < 0:
                continue
            room = table.shape[1] * P
            at = min(at, room)
            tree = None if parents is None else parents[b]
            deep = depths(tree, n)
            for i in range(n):
                nodes = path(tree, i)[::-1] if tree is not None else range(i + 1)
                places = [(p, p) for p in range(at)] + [(at + m, at + int(deep[m])) for m in nodes]
                mine = at + int(deep[i])
                seen = []
                for p, where in places:
                    s = slot(table, b, p, P, pages) if p < room else None
                    if s is not None and (window == 0 or mine - where < window):
                        seen.append((*s, mine - where))
                if not seen:
                    continue
                page, row, far = (np.array(x) for x in zip(*seen))
                for h in range(Hq):
                    k, v = cache["k"][page, row, h // G], cache["v"][page, row, h // G]
                    z = (k @ q[b, i, h]) * sm
                    smax[b, i, h] = np.abs(sm) * (np.abs(k) @ np.abs(q[b, i, h])).max()
                    if cap > 0:
                        z = cap * np.tanh(z / cap)
                    if slopes is not None:
                        z = z - slopes[h] * far
                    m = z.max()
                    e = np.exp(z - m)
                    lse[b, i, h] = m + np.log(e.sum())
                    zmax[b, i, h] = np.abs(z).max()
                    count[b, i, h] = len(z)
                    out[b, i, h] = (e / e.sum()) @ v
                    absv[b, i, h] = (e / e.sum()) @ np.abs(v)
    return out, lse, absv, smax, zmax, count
