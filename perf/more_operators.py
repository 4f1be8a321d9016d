"""The 16-bit paged cache's operators of a verify step: cases, inputs, plain forms and 64-bit values.

Two kinds of case, each one call as a serving loop makes it for one layer:

  append     new keys and values written into the cache, keys and queries rotated by position (spec_kv_append_rope)
  attention  the new rows' attention over that cache: chains, draft trees or prompts, scores capped by a tanh, a sliding
             window, a bias by distance (spec_attention)

A cache is k, v [pages, page size, kv heads, head dim] in the rows' type; slot p of request b is row p % page size of page
table[b, p / page size]. Row n of request b goes to slot base[b] + n; its position is that in a chain or prompt, and
base[b] plus its depth in a draft tree. An append returns the cache's own buffers; a pass over a state that an earlier
pass has written gives the same result again.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a verify step's six rows (five drafts and the root) of 32 requests
        dict(name="append_chain", kind="append", B=32, N=6, Hq=32, Hkv=8, D=128, P=16, L=4096, ragged=True, tree=False,
             rot=128, interleaved=False, dtype="bf16"),
        # 64-node draft trees far into long contexts; only a part of each head is rotated, in neighbouring pairs
        dict(name="append_tree", kind="append", B=16, N=64, Hq=64, Hkv=8, D=64, P=32, L=16384, ragged=True, tree=True,
             rot=32, interleaved=True, dtype="f16"),
        # three prompts enter the cache; a length that ends inside a page
        dict(name="append_prompt", kind="append", B=3, N=4099, Hq=32, Hkv=8, D=128, P=64, L=0, ragged=False, tree=False,
             rot=128, interleaved=False, dtype="bf16"),
        # one request, one token: latency
        dict(name="attention_decode", kind="attention", B=1, N=1, Hkv=8, G=4, D=128, P=16, L=1000, ragged=False, tree=False,
             cap=0.0, window=0, slopes=False, dtype="bf16"),
        # one token each for 64 requests of mixed lengths
        dict(name="attention_batch", kind="attention", B=64, N=1, Hkv=8, G=4, D=128, P=16, L=8192, ragged=True, tree=False,
             cap=0.0, window=0, slopes=False, dtype="bf16"),
        # verification of five drafts for 32 requests of mixed lengths, capped scores
        dict(name="attention_chain_cap", kind="attention", B=32, N=6, Hkv=8, G=4, D=128, P=16, L=8192, ragged=True,
             tree=False, cap=30.0, window=0, slopes=False, dtype="bf16"),
        # the same step in a layer with a sliding window, over long contexts, 64-wide heads
        dict(name="attention_window", kind="attention", B=16, N=6, Hkv=8, G=8, D=64, P=32, L=65536, ragged=True, tree=False,
             cap=0.0, window=4096, slopes=False, dtype="f16"),
        # a model that knows positions by a bias alone, every query head with keys of its own
        dict(name="attention_slopes", kind="attention", B=8, N=4, Hkv=32, G=1, D=128, P=16, L=4096, ragged=True, tree=False,
             cap=0.0, window=0, slopes=True, dtype="bf16"),
        # verification of 64-node draft trees, depth 5, for 16 requests
        dict(name="attention_tree", kind="attention", B=16, N=64, Hkv=8, G=4, D=128, P=64, L=8192, ragged=True, tree=True,
             cap=0.0, window=0, slopes=False, dtype="bf16"),
        # draft trees with capped scores and a window
        dict(name="attention_tree_cap", kind="attention", B=16, N=64, Hkv=8, G=4, D=128, P=64, L=8192, ragged=True,
             tree=True, cap=50.0, window=4096, slopes=False, dtype="bf16"),
        # a piece of a prompt after what the cache already holds of it, an odd number of rows
        dict(name="attention_piece", kind="attention", B=4, N=1001, Hkv=8, G=8, D=64, P=32, L=12000, ragged=True, tree=False,
             cap=0.0, window=0, slopes=False, dtype="f16"),
        # two whole prompts
        dict(name="attention_prompt", kind="attention", B=2, N=4099, Hkv=8, G=4, D=128, P=64, L=0, ragged=False, tree=False,
             cap=0.0, window=0, slopes=False, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


_MOST = {}


def _fits(case):
    """Whether a case costs no more than the largest listed one of its kind."""
    if not _MOST:
        for c in listed():
            w = work(c)
            m = _MOST.setdefault(c["kind"], {"bytes": 0, "flops": 0})
            m["bytes"], m["flops"] = max(m["bytes"], w["bytes"]), max(m["flops"], w["flops"])
    w, m = work(case), _MOST[case["kind"]]
    return w["bytes"] <= m["bytes"] and w["flops"] <= m["flops"] and case["B"] * (case["L"] + case["N"]) <= 64 * 8193


def draw(rng):
    while True:
        kind = rng.choice(["append", "attention", "attention"])
        tree = rng.random() < 0.3
        c = dict(kind=kind, B=_log_int(rng, 1, 64), D=rng.choice([64, 128]), P=rng.choice([16, 32, 64, 128]),
                 Hkv=rng.choice([1, 2, 4, 8, 16]), L=rng.choice([0, 1, 1, 1, 1, 1]) * _log_int(rng, 1, 65536),
                 ragged=rng.random() < 0.7, tree=tree,
                 N=rng.randint(2, 64) if tree else rng.choice([_log_int(rng, 1, 8), _log_int(rng, 1, 4500)]),
                 dtype=rng.choice(["bf16", "f16"]))
        G = rng.choice([1, 2, 4, 7, 8])
        if kind == "append":
            c.update(Hq=c["Hkv"] * G, rot=16 * rng.randint(1, c["D"] // 16) if rng.random() < 0.3 else c["D"],
                     interleaved=rng.random() < 0.4)
        else:
            c.update(G=G, cap=rng.choice([0.0, 0.0, 30.0, 50.0]), window=rng.choice([0, 0, _log_int(rng, 1, 8192)]),
                     slopes=rng.random() < 0.25)
        if _fits(c):
            return c


def _lengths(c):
    """Lengths below a request's new rows: spread over [L / 4, L] where they are ragged."""
    if not c["ragged"]:
        return [c["L"]] * c["B"]
    return [c["L"] - (c["L"] - c["L"] // 4) * i // max(1, c["B"] - 1) for i in range(c["B"])]


def work(case):
    """What one pass cannot do without: of the cache, the positions that a row sees."""
    c = case
    B, N, D = c["B"], c["N"], c["D"]
    if c["kind"] == "append":
        heads = 2 * c["Hkv"] + c["Hq"]
        return {"bytes": 4 * B * N * heads * D, "flops": 3 * B * N * (c["Hkv"] + c["Hq"]) * c["rot"]}
    seen = read = 0
    for base in _lengths(c):
        w = c["window"] or base + N
        read += min(base + N, w + N - 1)
        if c["tree"]:  # the prefix, and a handful of ancestors
            seen += N * (min(base, w) + min(3, w))
        else:  # row n sees min(base + n + 1, w) positions
            full = max(0, min(N, w - base))  # rows whose window reaches to the start
            seen += full * base + full * (full + 1) // 2 + (N - full) * w
    Hq = c["Hkv"] * c["G"]
    return {"bytes": 4 * c["Hkv"] * read * D + 4 * B * N * Hq * D, "flops": 4 * Hq * seen * D}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(shape, dtype, g, scale=1.0):
    """N(0, scale^2) in `dtype`, made in pieces of the first dimension."""
    out = torch.empty(shape, dtype=dtype, device="cuda")
    step = max(1, (1 << 27) // max(1, out[0].numel()))
    for i in range(0, shape[0], step):
        n = min(step, shape[0] - i)
        out[i:i + n] = (torch.randn((n, *shape[1:]), generator=g, device="cuda") * scale).to(dtype)
    return out


def _tree_parents(B, N, g):
    """Draft trees of depth below 6: node n's parent is an earlier node of depth below 5, the earlier the likelier."""
    u = torch.rand((B, N), generator=g, device="cuda").cpu().tolist()
    parents = []
    for b in range(B):
        par, depth, open_ = [-1], [0], [0]
        for n in range(1, N):
            p = open_[int(u[b][n] ** 1.5 * len(open_))]
            par.append(p)
            depth.append(depth[p] + 1)
            if depth[n] < 5:
                open_.append(n)
        parents.append(par)
    return torch.tensor(parents, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    c, g = case, _gen(seed)
    B, N, H, D, P, dt = c["B"], c["N"], c["Hkv"], c["D"], c["P"], DTYPES[c["dtype"]]
    order = torch.randperm(B, generator=g, device="cuda").cpu()
    base = torch.tensor(_lengths(c))[order].cuda()  # lengths in an order that goes by the seed
    need = (base + N + P - 1) // P
    total = int(need.sum())
    W = int(need.max())
    has = torch.arange(W, device="cuda")[None] < need[:, None]
    table = torch.full((B, W), -1, dtype=torch.int64, device="cuda")
    table[has] = torch.randperm(total, generator=g, device="cuda")  # a pool of shuffled pages
    Hq = c["Hq"] if c["kind"] == "append" else H * c["G"]
    s = dict(case=dict(c), k=_normal((total, P, H, D), dt, g), v=_normal((total, P, H, D), dt, g), table=table.to(torch.int32),
             base=base.to(torch.int32), parents=_tree_parents(B, N, g) if c["tree"] else None)
    if c["kind"] == "append":
        s.update(k_new=_normal((B, N, H, D), dt, g), v_new=_normal((B, N, H, D), dt, g), q=_normal((B, N, Hq, D), dt, g),
                 inv_freq=(500000.0 ** (-torch.arange(c["rot"] // 2, dtype=torch.float64, device="cuda") * 2 / c["rot"])).float())
    else:
        # rows whose scores have a spread of about 2, and of 8 where a cap bounds them
        s.update(q=_normal((B, N, Hq, D), dt, g, 8.0 if c["cap"] else 2.0), sm=1.0 / math.sqrt(D), slopes=None)
        if c["slopes"]:
            s["slopes"] = torch.exp2(-8.0 * torch.arange(1, Hq + 1, device="cuda") / Hq)
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import speculative_decoding_verification_72_gb300 as sv

    c, cache = s["case"], sv.PagedCache(s["k"], s["v"])
    if c["kind"] == "append":
        r = sv.spec_kv_append_rope(cache, s["k_new"], s["v_new"], s["table"], s["base"], s["inv_freq"], q=s["q"],
                                   parents=s["parents"], interleaved=c["interleaved"])
        return dict(k=s["k"], v=s["v"], q=r["q"], out_len=r["out_len"])
    r = sv.spec_attention(s["q"], cache, s["table"], s["base"], parents=s["parents"], sm_scale=s["sm"], softcap=c["cap"],
                          window=c["window"], slopes=s["slopes"])
    return dict(out=r["out"], lse=r["lse"])


def _run_plain(s):
    return _plain_append(s) if s["case"]["kind"] == "append" else _plain_attention(s)


# ------------------------------------------------------------------ plain forms

def _depths(s):
    """[B, N]: a row's position past its request's base."""
    c = s["case"]
    n = torch.arange(c["N"], device=s["k"].device)
    if s["parents"] is None:
        return n[None].expand(c["B"], -1)
    at, depth = s["parents"].long(), torch.zeros((c["B"], c["N"]), dtype=torch.int64, device=s["k"].device)
    for _ in range(5):
        depth += at >= 0
        at = torch.where(at >= 0, s["parents"].long().gather(1, at.clamp(min=0)), -1)
    return depth


def _turned(x, cos, sin, rot, interleaved):
    """x [B, N, heads, D] rotated by angles [B, N, 1, rot / 2], in 32 bits, rounded once."""
    y = x.float()
    if interleaved:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, y[..., rot:]], -1).to(x.dtype)


def _plain_append(s):
    c = s["case"]
    N, P = c["N"], c["P"]
    angle = (s["base"].long()[:, None] + _depths(s)).double()[..., None, None] * s["inv_freq"].double()  # far positions
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    slot = s["base"].long()[:, None] + torch.arange(N, device=s["k"].device)
    page = s["table"].long().gather(1, slot // P)
    s["k"][page, slot % P] = _turned(s["k_new"], cos, sin, c["rot"], c["interleaved"])
    s["v"][page, slot % P] = s["v_new"]
    return dict(k=s["k"], v=s["v"], q=_turned(s["q"], cos, sin, c["rot"], c["interleaved"]), out_len=s["base"] + N)


def _visible(s, lo, hi, S, depth):
    """([b, N, S] what rows of requests lo .. hi - 1 see, [b, S] positions of the slots)."""
    c, dev = s["case"], s["k"].device
    N, base = c["N"], s["base"].long()[lo:hi, None]
    j = torch.arange(S, device=dev)[None] - base  # slot, as a new row
    depth = depth[lo:hi]
    i = torch.arange(N, device=dev)
    if s["parents"] is None:
        see = j[:, None] <= i[None, :, None]
        position = (base + j).expand(-1, S)
    else:
        par = s["parents"].long()[lo:hi]
        up = torch.zeros((hi - lo, N, N + 1), device=dev).scatter_(2, torch.where(par < 0, N, par)[..., None], 1.0)[..., :N]
        up = up + torch.eye(N, device=dev)
        for _ in range(3):
            up = (up @ up > 0).float()  # ancestors up to eight levels above
        at = j.clamp(0, N - 1)
        see = (j[:, None] < 0) | ((j[:, None] < N) & (torch.gather(up, 2, at[:, None].expand(-1, N, -1)) > 0))
        position = torch.where(j < 0, base + j, base + depth.gather(1, at))
    if c["window"]:
        see = see & ((base + depth)[:, :, None] - position[:, None] < c["window"])
    return see, position


def _plain_attention(s):
    c = s["case"]
    B, N, H, G, D, P = c["B"], c["N"], c["Hkv"], c["G"], c["D"], c["P"]
    out = torch.empty_like(s["q"])
    lse = torch.empty((B, N, H * G), device=out.device)
    depth = _depths(s)
    S = s["table"].shape[1] * P
    step = max(1, (1 << 29) // (H * G * N * S))  # requests at a time: 2 GiB of scores
    for lo in range(0, B, step):
        hi = min(B, lo + step)
        page = s["table"].long()[lo:hi].clamp(min=0)
        k, v = (t[page].float().view(hi - lo, S, H, D).transpose(1, 2) for t in (s["k"], s["v"]))  # [b, H, S, D]
        q = s["q"][lo:hi].float().view(hi - lo, N, H, G, D).permute(0, 2, 1, 3, 4).reshape(hi - lo, H, N * G, D)
        x = ((q @ k.transpose(2, 3)) * s["sm"]).view(hi - lo, H, N, G, S)
        if c["cap"]:
            x = c["cap"] * torch.tanh(x / c["cap"])
        see, position = _visible(s, lo, hi, S, depth)
        if s["slopes"] is not None:
            far = (s["base"].long()[lo:hi, None] + depth[lo:hi])[:, :, None] - position[:, None]  # [b, N, S]
            x = x - s["slopes"].view(1, H, 1, G, 1) * far.float()[:, None, :, None]
        x = x.masked_fill(~see[:, None, :, None], -math.inf).view(hi - lo, H, N * G, S)
        m = x.amax(-1, keepdim=True)
        p = torch.exp(x - m)
        total = p.sum(-1, keepdim=True)
        o = (p @ v) / total
        out[lo:hi] = o.view(hi - lo, H, N, G, D).permute(0, 2, 1, 3, 4).reshape(hi - lo, N, H * G, D).to(out.dtype)
        lse[lo:hi] = (m + torch.log(total)).view(hi - lo, H, N, G).permute(0, 2, 1, 3).reshape(hi - lo, N, H * G)
    return dict(out=out, lse=lse)


# ------------------------------------------------------------------ 64-bit values

def exact(case, seed):
    s = prepare(case, seed)
    return _exact_append(s) if case["kind"] == "append" else _exact_attention(s)


def _paths(s, b):
    """For each new row of request b, the rows on its way up, itself first."""
    N = s["case"]["N"]
    par = s["parents"][b].tolist()
    paths = []
    for n in range(N):
        path = [n]
        while par[path[-1]] >= 0:
            path.append(par[path[-1]])
        paths.append(path)
    return paths


def _exact_append(s):
    c = s["case"]
    N, P, rot = c["N"], c["P"], c["rot"]
    got = dict(k=s["k"].double(), v=s["v"].double(), q=s["q"].double(), out_len=s["base"] + N)
    half = torch.arange(rot // 2, device=s["k"].device)
    first, second = (2 * half, 2 * half + 1) if c["interleaved"] else (half, half + rot // 2)
    for b, base in enumerate(s["base"].tolist()):
        deep = torch.arange(N) if s["parents"] is None else torch.tensor([len(p) - 1 for p in _paths(s, b)])
        turn = torch.polar(torch.ones((), dtype=torch.float64, device=half.device),
                           (base + deep.cuda()).double()[:, None, None] * s["inv_freq"].double())
        for x, to in ((s["k_new"][b].double(), None), (got["q"][b], got["q"][b])):
            z = torch.complex(x[..., first], x[..., second]) * turn
            y = x.clone()
            y[..., first], y[..., second] = z.real, z.imag
            if to is not None:
                to.copy_(y)
            else:
                for p in range(base // P, (base + N - 1) // P + 1):  # a page at a time
                    lo, hi, page = max(base, p * P), min(base + N, (p + 1) * P), int(s["table"][b, p])
                    got["k"][page, lo - p * P:hi - p * P] = y[lo - base:hi - base]
                    got["v"][page, lo - p * P:hi - p * P] = s["v_new"][b, lo - base:hi - base].double()
    return got


def _exact_attention(s):
    c = s["case"]
    B, N, H, G, D, P = c["B"], c["N"], c["Hkv"], c["G"], c["D"], c["P"]
    dev = s["k"].device
    out = torch.empty((B, N, H, G, D), dtype=torch.float64, device=dev)
    lse = torch.empty((B, N, H, G), dtype=torch.float64, device=dev)
    for b, base in enumerate(s["base"].tolist()):
        n = base + N
        spot = torch.arange(n, device=dev)
        if s["parents"] is None:
            deep, hidden = torch.arange(N, device=dev), spot[None] > base + torch.arange(N, device=dev)[:, None]
        else:
            paths = _paths(s, b)
            deep = torch.tensor([len(p) - 1 for p in paths], device=dev)
            hidden = torch.ones((N, n), dtype=torch.bool)
            hidden[:, :base] = False
            for i, p in enumerate(paths):
                hidden[i, [base + a for a in p]] = False
            hidden = hidden.to(dev)
        where = torch.cat([spot[:base], base + deep])
        far = ((base + deep)[:, None] - where[None]).double()
        if c["window"]:
            hidden = hidden | (far >= c["window"])
        pages = s["table"][b, :-(-n // P)].long()
        for h in range(H):
            k, v = (t[pages, :, h].reshape(-1, D)[:n].double() for t in (s["k"], s["v"]))
            for g in range(G):
                x = s["q"][b, :, h * G + g].double() @ k.T * s["sm"]
                if c["cap"]:
                    x = torch.tanh(x / c["cap"]) * c["cap"]
                if s["slopes"] is not None:
                    x = x - float(s["slopes"][h * G + g]) * far
                x = x.masked_fill(hidden, -math.inf)
                t = torch.logsumexp(x, -1)
                lse[b, :, h, g] = t
                out[b, :, h, g] = torch.exp(x - t[:, None]) @ v
    return dict(out=out.view(B, N, H * G, D), lse=lse.view(B, N, H * G))
