"""The verify step's cache, attention, eviction and log-prob operators: cases, inputs, plain forms and 64-bit values.

Five kinds of case, each one call (a training step: two) as a serving or training loop makes it:

  append     node or prompt rows written into a paged 8-bit cache (spec_kv_append_q8)
  attention  the verify pass's attention over that cache, chain or tree mask (spec_attention_q8)
  weights    accumulated attention weight of the accepted rows (spec_attention_weights_q8)
  evict      down to a budget by accumulated weight (spec_kv_evict_q8)
  logprobs   log-probs of given tokens, entropy, top alternatives; with the gradient where "train" is true
             (spec_token_logprobs, spec_token_logprobs_backward)

A cache is k, v in e4m3 [pages, kv heads, page size, head dim] with fp32 scales [pages, kv heads]; position p of
request b is slot p % page size of page table[b, p // page size]. Operators that change a cache return its buffers:
codes in a floating type of 8 bits, and their scales, whose products are the values. A pass over a state that an
earlier pass has written gives the same result again (the same rows to the same slots, and scales that have grown
already).
"""

import math

import torch

own = False

E4M3_MAX = 448.0
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a verify step's six rows (five drafts and the root) of 32 requests, for one layer's cache
        dict(name="append_chain", kind="append", B=32, N=6, Hkv=8, D=128, P=16, L=4096, ragged=True, dtype="bf16"),
        # three prompts enter the cache; a length that ends inside a page
        dict(name="append_prompt", kind="append", B=3, N=4099, Hkv=8, D=128, P=64, L=0, ragged=False, dtype="bf16"),
        # one request, one token: latency
        dict(name="attention_decode", kind="attention", B=1, N=1, Hkv=8, G=4, D=128, P=16, L=1000, ragged=False,
             tree=False, dtype="bf16"),
        # verification of five drafts for 32 requests of mixed lengths
        dict(name="attention_chain", kind="attention", B=32, N=6, Hkv=8, G=4, D=128, P=16, L=8192, ragged=True,
             tree=False, dtype="bf16"),
        # verification of 64-node draft trees, depth 5, for 16 requests
        dict(name="attention_tree", kind="attention", B=16, N=64, Hkv=8, G=4, D=128, P=64, L=8192, ragged=True,
             tree=True, dtype="bf16"),
        # the accepted rows of a small batch
        dict(name="weights_small", kind="weights", B=4, N=4, Hkv=8, G=4, D=128, P=16, L=700, ragged=True, dtype="bf16"),
        # the accepted rows over long contexts, 64-wide heads
        dict(name="weights_long", kind="weights", B=8, N=6, Hkv=8, G=8, D=64, P=32, L=65536, ragged=True, dtype="f16"),
        # two requests a little over their budget, as after each step of a bounded cache
        dict(name="evict_step", kind="evict", B=2, Hkv=8, D=128, P=16, L=1090, ragged=False, keep=1024),
        # 24 long prompts cut down to a budget after prefill
        dict(name="evict_prompt", kind="evict", B=24, Hkv=8, D=128, P=16, L=8192, ragged=True, keep=4096),
        # what a server returns beside the tokens of a verify step: 192 rows, 20 alternatives each
        dict(name="logprobs_serve", kind="logprobs", B=32, R=6, V=128256, n_top=20, masked=True, train=False, T=1.0,
             dtype="bf16"),
        # a training step on log-probs and entropy, odd vocabulary
        dict(name="logprobs_train_bf16", kind="logprobs", B=8, R=256, V=50257, n_top=0, masked=False, train=True, T=1.0,
             dtype="bf16"),
        # the same over a large vocabulary in 32 bits, at a sampling temperature
        dict(name="logprobs_train_f32", kind="logprobs", B=16, R=128, V=151936, n_top=0, masked=False, train=True, T=0.7,
             dtype="f32"),
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
    return w["bytes"] <= m["bytes"] and w["flops"] <= max(m["flops"], 1)


def draw(rng):
    while True:
        kind = rng.choice(["append", "attention", "attention", "weights", "evict", "logprobs", "logprobs"])
        c = dict(kind=kind)
        if kind == "logprobs":
            train = rng.random() < 0.5
            c.update(B=_log_int(rng, 1, 64), R=_log_int(rng, 1, 256), V=_log_int(rng, 1000, 160000),
                     n_top=0 if train else rng.choice([0, 1, 5, 20, 32]), masked=rng.random() < 0.5, train=train,
                     T=rng.choice([1.0, 0.7, 1.3]), dtype=rng.choice(["bf16", "f32"]))
        else:
            c.update(B=_log_int(rng, 1, 48), Hkv=rng.choice([1, 2, 4, 8]), D=rng.choice([64, 128]),
                     P=rng.choice([16, 32, 64, 128]), L=_log_int(rng, 1, 65536), ragged=rng.random() < 0.7)
            if kind == "append":
                c.update(N=_log_int(rng, 1, 4096), dtype=rng.choice(["bf16", "f16", "f32"]))
            elif kind == "attention":
                tree = rng.random() < 0.4
                c.update(N=rng.randint(8, 64) if tree else rng.randint(1, 8), G=rng.choice([1, 2, 4, 8]), tree=tree,
                         dtype=rng.choice(["bf16", "f16"]))
            elif kind == "weights":
                c.update(N=rng.randint(1, 8), G=rng.choice([1, 2, 4, 8]), dtype=rng.choice(["bf16", "f16"]))
            else:
                c.update(L=_log_int(rng, 200, 32768))
                c.update(keep=max(1, int(c["L"] * rng.uniform(0.3, 0.97)) // c["P"]) * c["P"])
        if _fits(c):
            return c


def work(case):
    """What one pass cannot do without. Ragged lengths are uniform over [L/4, L], so L counts as 5/8 of it."""
    c, kind = case, case["kind"]
    if kind == "logprobs":
        es, n = (4 if c["dtype"] == "f32" else 2), c["B"] * c["R"] * c["V"]
        return {"bytes": n * es * (2 if c["train"] else 1), "flops": n * (10 if c["train"] else 5)}
    B, H, D = c["B"], c["Hkv"], c["D"]
    L = c["L"] * 0.625 if c["ragged"] else c["L"]
    if kind == "append":
        es = 4 if c["dtype"] == "f32" else 2
        return {"bytes": 2 * B * c["N"] * H * D * (es + 1), "flops": 4 * B * c["N"] * H * D}
    if kind == "evict":
        moved = B * H * c["keep"] * max(0.0, 1 - c["keep"] / max(L, c["keep"]))
        return {"bytes": 16 * B * H * L + 4 * D * moved, "flops": 2 * D * moved + 8 * B * H * L}
    rows = B * c["N"] * H * c["G"]
    L += c["N"]
    if kind == "attention":
        return {"bytes": 2 * B * H * L * D + 4 * rows * D, "flops": 4 * rows * L * D}
    return {"bytes": B * H * L * (D + 8) + 2 * rows * D, "flops": 2 * rows * L * D}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _codes(pages, H, P, D, g):
    """Codes of rows with entries N(0, 1) under a scale of 2^-7 or so: magnitudes up to the type's largest."""
    out = torch.empty((pages, H, P, D), dtype=torch.float8_e4m3fn, device="cuda")
    step = max(1, (1 << 27) // (H * P * D))
    for i in range(0, pages, step):
        n = min(step, pages - i)
        out[i:i + n] = (torch.randn((n, H, P, D), generator=g, device="cuda") * 100).clamp_(-448, 448).to(out.dtype)
    return out


def _tree_parents(B, N, g):
    """Draft trees of up to 64 nodes and depth 5: node n's parent is an earlier node of depth below 5, the earlier the likelier."""
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


def _cache(c, extra, g):
    """A pool of shuffled pages that holds each request's positions and `extra` more; (state, base, S)."""
    B, H, P, D, L = c["B"], c["Hkv"], c["P"], c["D"], c["L"]
    if c["ragged"]:  # lengths spread over [L / 4, L], in an order that goes by the seed
        base = L - (L - L // 4) * torch.randperm(B, generator=g, device="cuda") // max(1, B - 1)
    else:
        base = torch.full((B,), L, device="cuda")
    W = max(1, -(-(L + extra) // P))
    need = (base + extra + P - 1) // P
    total = int(need.sum())
    ids = torch.randperm(total, generator=g, device="cuda")
    has = torch.arange(W, device="cuda")[None] < need[:, None]
    table = torch.full((B, W), -1, dtype=torch.int64, device="cuda")
    table[has] = ids
    scale = lambda: torch.exp2(torch.randint(-8, -5, (total + 1, H), generator=g, device="cuda").float())  # noqa: E731
    s = dict(k=_codes(total + 1, H, P, D, g), v=_codes(total + 1, H, P, D, g), k_scale=scale(), v_scale=scale(),
             table=table.to(torch.int32), base=base.to(torch.int32))
    return s, W * P


def _positions(n, H, S, g):
    """Token positions that the slots hold: those of slots below n are the numbers below n, in another order for each head."""
    u = torch.rand((n.shape[0], H, S), generator=g, device="cuda")
    u.masked_fill_(torch.arange(S, device="cuda") >= n[:, None, None], 2.0)
    return u.argsort(-1).argsort(-1).to(torch.int32)


def prepare(case, seed):
    c, g = case, _gen(seed)
    kind = c["kind"]
    s = dict(case=dict(c))
    if kind == "logprobs":
        B, R, V, dt = c["B"], c["R"], c["V"], DTYPES[c["dtype"]]
        x = torch.empty((B, R, V), dtype=dt, device="cuda")
        for b in range(B):
            x[b] = (torch.randn((R, V), generator=g, device="cuda") * 3).to(dt)
        if c["masked"]:  # a grammar or a stop set masks some tokens
            for b in range(B):
                x[b].masked_fill_(torch.rand((R, V), generator=g, device="cuda") < 0.1, -math.inf)
        s.update(x=x, tokens=torch.randint(0, V, (B, R), generator=g, device="cuda", dtype=torch.int32))
        if c["train"]:
            s["tokens"][:, -1:] = -1  # padding at the end of each sequence
            s.update(x=x.nan_to_num_(neginf=-30.0), g_lp=torch.randn((B, R), generator=g, device="cuda"),
                     g_ent=0.01 * torch.randn((B, R), generator=g, device="cuda"))
    elif kind == "evict":
        B, H = c["B"], c["Hkv"]
        cache, S = _cache(c, 0, g)
        s.update(cache)
        # weight accumulates over a slot's life and is heavy-tailed; slots hold tokens in no particular order
        age = 1 - torch.arange(S, device="cuda") / S
        s.update(S=S, keep=c["keep"], sinks=4,
                 scores=torch.exp(2 * torch.randn((B, H, S), generator=g, device="cuda")) * age,
                 positions=_positions(s["base"], H, S, g))
        s["protect_from"] = s["base"].clone()
        s["protect_from"].sub_(c["keep"] // 16)
    else:
        B, N, H, D, dt = c["B"], c["N"], c["Hkv"], c["D"], DTYPES[c["dtype"]]
        cache, S = _cache(c, N, g)
        s.update(cache, S=S)
        if kind == "append":
            s.update(k_new=torch.randn((B, N, H, D), generator=g, device="cuda").to(dt),
                     v_new=torch.randn((B, N, H, D), generator=g, device="cuda").to(dt))
        else:
            # rows whose scores have a spread of about 2
            s["q"] = (torch.randn((B, N, H * c["G"], D), generator=g, device="cuda") * 2).to(dt)
            s["sm"] = 1.0 / math.sqrt(D)
            if kind == "attention":
                s["parents"] = _tree_parents(B, N, g) if c["tree"] else None
            else:  # the first accepted rows of the verify pass
                s["n_acc"] = torch.randint(0, N, (B,), generator=g, device="cuda", dtype=torch.int32)
                s["path"] = (torch.rand((B, N - 1), generator=g, device="cuda").argsort(-1) + 1).to(torch.int32)
                s["path"] = torch.cat([torch.zeros_like(s["table"][:, :1]), s["path"].sort(-1).values], 1).contiguous()
                s["scores"] = torch.rand((B, H, S), generator=g, device="cuda")
                s["lse"] = torch.zeros((B, N, H * c["G"]), device="cuda")
                _plain_weights(s, lse_only=True)
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import speculative_decoding_verification_72_gb300 as sv

    kind = s["case"]["kind"]
    cache = None if kind == "logprobs" else sv.Q8Cache(s["k"], s["v"], s["k_scale"], s["v_scale"])
    if kind == "append":
        r = sv.spec_kv_append_q8(cache, s["k_new"], s["v_new"], s["table"], s["base"])
        return _cache_out(s, out_len=r["out_len"])
    if kind == "attention":
        r = sv.spec_attention_q8(s["q"], cache, s["table"], s["base"], parents=s["parents"], sm_scale=s["sm"])
        return dict(out=r["out"], lse=r["lse"])
    if kind == "weights":
        r = sv.spec_attention_weights_q8(s["q"], s["lse"], cache, s["table"], s["base"], s["scores"],
                                         path_nodes=s["path"], num_accepted=s["n_acc"], sm_scale=s["sm"], decay=0.95)
        return dict(scores=r["scores"])
    if kind == "evict":
        r = sv.spec_kv_evict_q8(cache, s["table"], s["base"], s["scores"], s["positions"], s["keep"],
                                sinks=s["sinks"], protect_from=s["protect_from"])
        return _cache_out(s, scores=r["scores"], positions=r["positions"], out_len=r["out_len"])
    c = s["case"]
    r = sv.spec_token_logprobs(s["x"], s["tokens"], temperature=c["T"], n_top=c["n_top"])
    got = dict(logprob=r["logprob"], entropy=r["entropy"], lse=r["lse"])
    if c["n_top"]:
        got.update(top_tokens=r["top_tokens"], top_logprobs=r["top_logprobs"])
    if c["train"]:
        got["grad"] = sv.spec_token_logprobs_backward(s["x"], s["tokens"], r["saved"], s["g_lp"], grad_entropy=s["g_ent"],
                                                      temperature=c["T"])
    return got


def _cache_out(s, **more):
    return dict(k=s["k"], v=s["v"], k_scale=s["k_scale"], v_scale=s["v_scale"], **more)


def _run_plain(s):
    return dict(append=_plain_append, attention=_plain_attention, weights=_plain_weights, evict=_plain_evict,
                logprobs=_plain_logprobs)[s["case"]["kind"]](s)


# ------------------------------------------------------------------ plain forms

def _need_scale(amax):
    """The smallest power of two s with amax <= 448 s, and no less than 2^-100."""
    m, e = torch.frexp(amax)  # amax = m 2^e with m in [0.5, 1); 448 = 0.875 * 2^9
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(-100, 119)
    return torch.where(amax > 0, torch.exp2(e.float()), torch.full_like(amax, 2.0 ** -100))


def _plain_append(s):
    c = s["case"]
    B, N, P, dev = c["B"], c["N"], c["P"], s["k"].device
    base = s["base"].long()
    first = base // P
    W = (N + P - 1) // P + 1  # pages that a request's rows can touch
    slot = first[:, None] * P + torch.arange(W * P, device=dev)  # positions of those pages [B, W P]
    row = slot - base[:, None]
    new, kept = (row >= 0) & (row < N), row < 0
    lp = (first[:, None] + torch.arange(W, device=dev)).clamp(max=s["table"].shape[1] - 1)
    page = s["table"].long().gather(1, lp)
    touched = new.view(B, W, P).any(-1)
    page = torch.where(touched, page, torch.full_like(page, s["k"].shape[0] - 1))  # the pool's spare page takes the rest
    row = row.clamp(0, N - 1)
    take = torch.arange(B, device=dev)[:, None]
    new5, kept5 = new.view(B, W, 1, P, 1), kept.view(B, W, 1, P, 1)
    spare = [t[-1].clone() for t in (s["k"], s["v"], s["k_scale"], s["v_scale"])]
    for codes, scales, x in ((s["k"], s["k_scale"], s["k_new"]), (s["v"], s["v_scale"], s["v_new"])):
        x = x.float()[take, row].view(B, W, P, c["Hkv"], c["D"]).transpose(2, 3)  # [B, W, H, P, D]
        need = _need_scale((x.abs() * new5).amax((-1, -2)))
        old = scales[page]
        scale = torch.where(kept.view(B, W, P).any(-1)[..., None], torch.maximum(need, old), need)
        was = codes[page]
        moved = (was.float() * (old / scale)[..., None, None]).to(codes.dtype)
        fresh = (x / scale[..., None, None]).clamp(-E4M3_MAX, E4M3_MAX).to(codes.dtype)
        codes[page] = torch.where(new5, fresh.float(), torch.where(kept5, moved.float(), was.float())).to(codes.dtype)
        scales[page] = torch.where(touched[..., None], scale, old)
    for t, was in zip((s["k"], s["v"], s["k_scale"], s["v_scale"]), spare):
        t[-1] = was
    return _cache_out(s, out_len=s["base"] + N)


def _dense(s, codes, scales):
    """[B, Hkv, S, D] of a cache's values in 32 bits."""
    page = s["table"].long()
    page = torch.where(page < 0, codes.shape[0] - 1, page)
    x = codes[page].float() * scales[page][..., None, None]
    return x.transpose(1, 2).reshape(x.shape[0], x.shape[2], -1, x.shape[4])


def _visible(s, rows):
    """[B, rows, S]: whether row i of a request, at position base + i, attends to position j."""
    S, N, dev = s["S"], rows, s["k"].device
    base = s["base"].long()[:, None, None]
    j = torch.arange(S, device=dev)[None, None] - base  # position within the request's new rows
    i = torch.arange(N, device=dev)[None, :, None]
    if s.get("parents") is None:
        return j <= i
    par = s["parents"].long()
    up = torch.zeros((par.shape[0], N, N + 1), device=dev).scatter_(2, torch.where(par < 0, N, par)[..., None], 1.0)[..., :N]
    up = up + torch.eye(N, device=dev)
    up = (up @ up > 0).float()
    up = (up @ up > 0).float()
    up = up @ up > 0  # ancestors up to eight levels above
    within = torch.gather(up, 2, j.clamp(0, N - 1).expand(-1, N, -1))
    return (j < 0) | ((j < N) & within)


def _scores_of(s, q, visible):
    """Scaled scores [B, Hkv, rows * G, S] of q [B, rows, Hq, D], -inf where not visible."""
    c = s["case"]
    B, n, G = q.shape[0], q.shape[1], c["G"]
    q = q.float().view(B, n, c["Hkv"], G, c["D"]).permute(0, 2, 1, 3, 4).reshape(B, c["Hkv"], n * G, c["D"])
    x = q @ _dense(s, s["k"], s["k_scale"]).transpose(2, 3) * s["sm"]
    x = x.view(B, c["Hkv"], n, G, -1).masked_fill_(~visible[:, None, :, None], -math.inf)
    return x.view(B, c["Hkv"], n * G, -1)


def _plain_attention(s):
    c = s["case"]
    B, N, H, G, D = c["B"], c["N"], c["Hkv"], c["G"], c["D"]
    x = _scores_of(s, s["q"], _visible(s, N))
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    o = (p @ _dense(s, s["v"], s["v_scale"])) / total
    lse = (m + torch.log(total)).view(B, H, N, G)
    return dict(out=o.view(B, H, N, G, D).permute(0, 2, 1, 3, 4).reshape(B, N, H * G, D).to(s["q"].dtype),
                lse=lse.permute(0, 2, 1, 3).reshape(B, N, H * G))


def _plain_weights(s, lse_only=False):
    c = s["case"]
    B, N, H, G = c["B"], c["N"], c["Hkv"], c["G"]
    take, path = torch.arange(B, device=s["q"].device)[:, None], s["path"].long()
    x = _scores_of(s, s["q"][take, path], _visible(s, N))
    if lse_only:  # prepare(): what the attention call has left for these rows
        lse = torch.logsumexp(x, -1).view(B, H, N, G).permute(0, 2, 1, 3).reshape(B, N, H * G)
        s["lse"][take, path] = lse
        return None
    lse = s["lse"][take, path].view(B, N, H, G).permute(0, 2, 1, 3).reshape(B, H, N * G, 1)
    counted = (torch.arange(N, device=x.device)[None] <= s["n_acc"][:, None]).float()
    w = (torch.exp(x - lse).view(B, H, N, G, -1) * counted[:, None, :, None, None]).sum((2, 3))
    j, base = torch.arange(s["S"], device=x.device)[None], s["base"].long()[:, None]
    before, live = (j < base)[:, None], (j <= base + s["n_acc"][:, None])[:, None]
    return dict(scores=torch.where(before, 0.95 * s["scores"] + w, torch.where(live, w, torch.zeros_like(w))))


def _ordered(x):
    """Whole numbers in [0, 2^32) in the order of the values of x in 32 bits."""
    i = (x.float() + 0.0).view(torch.int32)
    return (i ^ ((i >> 31) & 0x7FFFFFFF)).long() + (1 << 31)


def _plain_evict(s):
    c = s["case"]
    B, H, P, D, S, keep, dev = c["B"], c["Hkv"], c["P"], c["D"], s["S"], s["keep"], s["k"].device
    n = s["base"].long()[:, None, None]
    slot = torch.arange(S, device=dev)
    valid = slot < n
    protected = (s["positions"] < s["sinks"]) | (s["positions"] >= s["protect_from"][:, None, None])
    key = torch.where(protected, 1 << 57, _ordered(s["scores"]) << 24) + (S - 1 - slot)
    key = torch.where(valid, key, -1 - slot)
    best = key.topk(min(keep, S), -1).indices
    kept = torch.zeros((B, H, S), dtype=torch.bool, device=dev).scatter_(2, best, True) & valid
    K = min(keep, S)
    hole, mover = valid[..., :K] & ~kept[..., :K], kept.clone()
    mover[..., :K] = False
    order = torch.where(mover, slot, S + slot).sort(-1).values  # movers first, ascending
    nth = (hole.long().cumsum(-1) - 1).clamp(min=0)
    src = torch.where(hole & (n > keep), order.gather(2, nth) % S, slot[:K])  # [B, H, K]
    spare = s["k"].shape[0] - 1
    table = torch.where(s["table"] < 0, spare, s["table"].long())
    page = table.gather(1, (src // P).view(B, -1)).view(B, H, K)
    head = torch.arange(H, device=dev)[None, :, None]
    to = table[:, None, :K // P].expand(B, H, K // P)
    for codes, scales in ((s["k"], s["k_scale"]), (s["v"], s["v_scale"])):
        from_scale = scales[page, head]
        scale = from_scale.view(B, H, K // P, P).amax(-1)
        x = codes[page, head, src % P].float() * (from_scale.view(B, H, K // P, P) / scale[..., None]).view(B, H, K, 1)
        was, was_scale = codes[spare].clone(), scales[spare].clone()
        codes[to, head] = x.view(B, H, K // P, P, D).to(codes.dtype)
        scales[to, head] = scale
        codes[spare], scales[spare] = was, was_scale
    out_len = s["base"].clamp(max=keep)
    live = slot < out_len[:, None, None]
    scores, positions = torch.zeros_like(s["scores"]), torch.full_like(s["positions"], -1)
    scores[..., :K] = s["scores"].gather(2, src)
    positions[..., :K] = s["positions"].gather(2, src)
    return _cache_out(s, scores=torch.where(live, scores, 0.0), positions=torch.where(live, positions, -1),
                      out_len=out_len)


def _plain_logprobs(s):
    c, x, tokens = s["case"], s["x"], s["tokens"].long()
    z = x.float() / c["T"]
    m = z.amax(-1, keepdim=True)
    e = torch.exp(z - m)
    total = e.sum(-1, keepdim=True)
    lse = m + torch.log(total)
    p = e / total
    ent = lse[..., 0] - torch.where(p > 0, p * z, 0.0).sum(-1)
    counted = tokens >= 0
    lp = torch.where(counted, z.gather(2, tokens.clamp(min=0)[..., None])[..., 0] - lse[..., 0], 0.0)
    got = dict(logprob=lp, entropy=ent, lse=lse[..., 0])
    if c["n_top"]:
        V = x.shape[-1]
        key = (_ordered(x) << 24) + (V - 1 - torch.arange(V, device=x.device))
        top = V - 1 - (key.topk(c["n_top"], -1).values & 0xFFFFFF)
        got.update(top_tokens=top.to(torch.int32), top_logprobs=z.gather(2, top) - lse)
    if c["train"]:
        g = torch.where(counted, s["g_lp"], 0.0)
        grad = p * (-g[..., None] - s["g_ent"][..., None] * (z - lse + ent[..., None]))
        grad.scatter_add_(2, tokens.clamp(min=0)[..., None], g[..., None])
        got["grad"] = (grad / c["T"]).to(x.dtype)
    return got


# ------------------------------------------------------------------ 64-bit values

def exact(case, seed):
    s = prepare(case, seed)
    return dict(append=_exact_append, attention=_exact_attention, weights=_exact_weights, evict=_exact_evict,
                logprobs=_exact_logprobs)[case["kind"]](s)


def _e4m3(x):
    """The nearest e4m3 value, ties to an even last bit, of float64 x with |x| <= 448."""
    _, e = torch.frexp(x)
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3)
    return torch.round(x / step) * step


def _values(s, b, h, n, codes, scales):
    P = s["case"]["P"]
    page = s["table"][b, :-(-n // P)].long()
    x = codes[page, h].double() * scales[page, h].double()[:, None, None]
    return x.reshape(-1, x.shape[-1])[:n]


def _exact_append(s):
    c = s["case"]
    N, P = c["N"], c["P"]
    got = {}
    for name, new in (("k", s["k_new"]), ("v", s["v_new"])):
        codes, scales = s[name].double(), s[name + "_scale"].double()
        for b, base in enumerate(s["base"].tolist()):
            for lp in range(base // P, (base + N - 1) // P + 1):
                lo, hi, page = max(base, lp * P), min(base + N, (lp + 1) * P), int(s["table"][b, lp])
                x = new[b, lo - base:hi - base].double().transpose(0, 1)  # [H, rows, D]
                e = torch.ceil(torch.log2(x.abs().amax((1, 2)) / E4M3_MAX))
                scale, kept = torch.exp2(e), lo - lp * P
                if kept:
                    scale = torch.maximum(scale, scales[page])
                    codes[page, :, :kept] = _e4m3(codes[page, :, :kept] * (scales[page] / scale)[:, None, None])
                codes[page, :, kept:hi - lp * P] = _e4m3(x / scale[:, None, None])
                scales[page] = scale
        got[name], got[name + "_scale"] = codes, scales
    return dict(got, out_len=s["base"] + N)


def _sees(s, b, rows, n):
    """Positions below n that each of a request's rows attends to, by walking up its tree."""
    base = int(s["base"][b])
    see = torch.zeros((rows, n), dtype=torch.bool)
    see[:, :base] = True
    par = s["parents"][b].tolist() if s.get("parents") is not None else list(range(-1, rows - 1))
    for i in range(rows):
        a = i
        while a >= 0:
            see[i, base + a] = True
            a = par[a]
    return see.cuda()


def _exact_attention(s):
    c = s["case"]
    B, N, H, G, D = c["B"], c["N"], c["Hkv"], c["G"], c["D"]
    out = torch.empty((B, N, H, G, D), dtype=torch.float64, device="cuda")
    lse = torch.empty((B, N, H, G), dtype=torch.float64, device="cuda")
    for b, base in enumerate(s["base"].tolist()):
        n = base + N
        see = _sees(s, b, N, n)
        for h in range(H):
            k, v = _values(s, b, h, n, s["k"], s["k_scale"]), _values(s, b, h, n, s["v"], s["v_scale"])
            x = torch.einsum("ngd,ld->ngl", s["q"].view(B, N, H, G, D)[b, :, h].double(), k) * s["sm"]
            x = x.masked_fill(~see[:, None], -math.inf)
            lse[b, :, h] = torch.logsumexp(x, -1)
            out[b, :, h] = torch.einsum("ngl,ld->ngd", torch.exp(x - lse[b, :, h][..., None]), v)
    return dict(out=out.view(B, N, H * G, D), lse=lse.view(B, N, H * G))


def _exact_weights(s):
    c = s["case"]
    H, G, D = c["Hkv"], c["G"], c["D"]
    scores = torch.zeros_like(s["scores"], dtype=torch.float64)
    for b, base in enumerate(s["base"].tolist()):
        n_rows = int(s["n_acc"][b]) + 1
        n, path = base + n_rows, s["path"][b, :n_rows].long()
        see = _sees(s, b, n_rows, n)
        for h in range(H):
            k = _values(s, b, h, n, s["k"], s["k_scale"])
            q = s["q"][b, path].view(n_rows, H, G, D)[:, h].double()
            x = torch.einsum("ngd,ld->ngl", q, k) * s["sm"] - s["lse"][b, path].view(n_rows, H, G)[:, h].double()[..., None]
            scores[b, h, :n] = torch.exp(x.masked_fill(~see[:, None], -math.inf)).sum((0, 1))
            scores[b, h, :base] += 0.95 * s["scores"][b, h, :base].double()
    return dict(scores=scores)


def _exact_evict(s):
    c = s["case"]
    P, keep = c["P"], s["keep"]
    got = {n: s[n].double() for n in ("k", "v", "k_scale", "v_scale")}
    scores, positions = torch.zeros_like(s["scores"], dtype=torch.float64), torch.full_like(s["positions"], -1)
    for b, n in enumerate(s["base"].tolist()):
        m = min(n, keep)
        scores[b, :, :m], positions[b, :, :m] = s["scores"][b, :, :m].double(), s["positions"][b, :, :m]
        if n <= keep:
            continue
        table = s["table"][b].long()
        for h in range(c["Hkv"]):
            pos, sc = s["positions"][b, h, :n], s["scores"][b, h, :n].double()
            rank = torch.where((pos < s["sinks"]) | (pos >= s["protect_from"][b]), math.inf, sc)
            kept = torch.zeros(n, dtype=torch.bool, device="cuda")
            kept[rank.sort(descending=True, stable=True).indices[:keep]] = True
            to, frm = (~kept[:keep]).nonzero()[:, 0], keep + kept[keep:].nonzero()[:, 0]
            src = torch.arange(keep, device="cuda")
            src[to] = frm
            scores[b, h, to], positions[b, h, to] = sc[frm], pos[frm]
            at, pages = table[src // P], table[:keep // P]
            for name in ("k", "v"):
                old = s[name + "_scale"][at, h].double()
                new = old.view(-1, P).max(1).values
                x = s[name][at, h, src % P].double() * (old / new.repeat_interleave(P))[:, None]
                got[name][pages, h] = _e4m3(x).view(-1, P, c["D"])
                got[name + "_scale"][pages, h] = new
    return dict(got, scores=scores, positions=positions, out_len=s["base"].clamp(max=keep))


def _exact_logprobs(s):
    c, tokens = s["case"], s["tokens"].long()
    B, R, V = s["x"].shape
    got = dict(logprob=torch.zeros((B, R), dtype=torch.float64, device="cuda"))
    got.update(entropy=got["logprob"].clone(), lse=got["logprob"].clone())
    if c["n_top"]:
        got.update(top_tokens=torch.zeros((B, R, c["n_top"]), dtype=torch.int32, device="cuda"))
        got.update(top_logprobs=torch.zeros((B, R, c["n_top"]), dtype=torch.float64, device="cuda"))
    if c["train"]:
        got["grad"] = torch.empty((B, R, V), dtype=torch.float64, device="cuda")
    for b in range(B):
        z = s["x"][b].double() / c["T"]
        lse = torch.logsumexp(z, -1)
        lp = z - lse[:, None]
        p = torch.exp(lp)
        ent = -torch.where(p > 0, p * lp, 0.0).sum(-1)
        given = torch.nn.functional.one_hot(tokens[b].clamp(min=0), V).bool() & (tokens[b] >= 0)[:, None]
        got["lse"][b], got["entropy"][b] = lse, ent
        got["logprob"][b] = torch.where(given, lp, 0.0).sum(-1)
        if c["n_top"]:
            at = s["x"][b].double().sort(dim=-1, descending=True, stable=True).indices[:, :c["n_top"]]
            got["top_tokens"][b], got["top_logprobs"][b] = at.to(torch.int32), lp.gather(1, at)
        if c["train"]:
            g, h = torch.where(tokens[b] >= 0, s["g_lp"][b].double(), 0.0)[:, None], s["g_ent"][b].double()[:, None]
            got["grad"][b] = (torch.where(given, g, 0.0) - g * p - h * p * (lp + ent[:, None])) / c["T"]
    return got
