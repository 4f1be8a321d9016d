"""spec_attention over the 16-bit paged cache against the oracle: both kernels, masks, caps, windows, biases."""

import numpy as np
import pytest
import torch

import speculative_decoding_verification_72_gb300 as sv
from oracle import kv_paged as K
from paged_utils import DEV, check_attention, host_cache, i32, normal, table, to_gpu, tree

pytestmark = pytest.mark.gpu

BF, F16 = torch.bfloat16, torch.float16


def run(rng, base, N, H, G, D, P, dtype, parents=None, n_nodes=None, sm=None, cap=0.0, window=0, slopes=None, layout="nhd", tab=None,
        pages=None, cache=None, q_std=2.0, q=None):
    B, sm = len(base), D ** -0.5 if sm is None else sm
    lens = [max(b, 0) + N for b in base]
    pages = pages or sum(-(-n // P) for n in lens) + 2
    tab = table(rng, lens, P, pages) if tab is None else tab
    c = host_cache(rng, pages, P, H, D, dtype) if cache is None else cache
    hq, gq = normal(rng, (B, N, H * G, D), dtype, q_std) if q is None else q
    r = sv.spec_attention(gq, to_gpu(c, dtype, layout), i32(tab), i32(base), parents=None if parents is None else i32(parents),
                          n_nodes=None if n_nodes is None else i32(n_nodes), sm_scale=sm, softcap=cap, window=window,
                          slopes=None if slopes is None else torch.tensor(slopes, dtype=torch.float32, device=DEV))
    want = K.attention(hq, c, tab, base, parents, n_nodes, sm, cap, window, slopes)
    check_attention(r, want, dtype, N * G, cap)
    return r, want


def slopes_of(Hq):
    return 2.0 ** (-8.0 * np.arange(1, Hq + 1) / Hq)


# ------------------------------------------------------- few rows a kv head

@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("D,P", [(128, 16), (64, 32), (64, 128), (128, 64)])
@pytest.mark.parametrize("N,G", [(1, 1), (1, 4), (3, 5), (6, 4), (1, 32), (16, 2), (32, 1)])
def test_few_rows(dtype, D, P, N, G):
    run(np.random.default_rng(N * G + D), [0, 1, 127, 128, 300], N, 2, G, D, P, dtype)


@pytest.mark.parametrize("N,G", [(2, 1), (8, 4), (20, 1), (5, 3)])
@pytest.mark.parametrize("D", [64, 128])
def test_few_rows_of_trees(N, G, D):
    rng = np.random.default_rng(N)
    run(rng, [0, 125, 40, 260], N, 2, G, D, 16, BF, parents=tree(rng, 4, N))


# ------------------------------------------------------- many rows a kv head

@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("D,P", [(128, 16), (64, 32), (64, 128), (128, 64)])
@pytest.mark.parametrize("N,G", [(33, 1), (9, 4), (70, 2), (43, 3), (130, 1)])
def test_many_rows(dtype, D, P, N, G):
    run(np.random.default_rng(N * G + D), [0, 1, 127, 300], N, 1, G, D, P, dtype)


@pytest.mark.parametrize("N,G", [(64, 4), (33, 1), (200, 2), (20, 7)])
@pytest.mark.parametrize("D", [64, 128])
def test_many_rows_of_trees(N, G, D):
    rng = np.random.default_rng(N)
    run(rng, [0, 125, 260], N, 1, G, D, 16, F16 if N == 200 else BF, parents=tree(rng, 3, N, 20 if N == 200 else 5))


def test_a_prompt_of_several_blocks():
    run(np.random.default_rng(8), [0, 77], 300, 1, 2, 64, 32, BF)


# ------------------------------------------------------- caps, windows, biases

@pytest.mark.parametrize("N,G", [(1, 4), (6, 5), (20, 4), (140, 2)])
@pytest.mark.parametrize("cap,window,bias", [(5.0, 0, False), (0.0, 40, False), (0.0, 0, True), (30.0, 130, True), (0.0, 1, False)])
def test_chain_variants(N, G, cap, window, bias):
    run(np.random.default_rng(N + window), [0, 90, 300], N, 2, G, 64, 16, BF, cap=cap, window=window,
        slopes=slopes_of(2 * G) if bias else None, q_std=8.0 if cap else 2.0)


@pytest.mark.parametrize("N,G", [(8, 3), (64, 4)])
@pytest.mark.parametrize("cap,window,bias", [(5.0, 0, False), (0.0, 3, False), (0.0, 0, True), (50.0, 129, True)])
def test_tree_variants(N, G, cap, window, bias):
    rng = np.random.default_rng(N + window)
    run(rng, [0, 126, 300], N, 1, G, 128, 16, F16, parents=tree(rng, 3, N), cap=cap, window=window,
        slopes=slopes_of(G) if bias else None, q_std=8.0 if cap else 2.0)


@pytest.mark.parametrize("N,G", [(33, 1), (20, 4), (16, 8)])
@pytest.mark.parametrize("window", [0, 100])
@pytest.mark.parametrize("D", [64, 128])
def test_biased_trees_whose_rows_share_tiles(N, G, window, D):
    """One tile, an even and an odd number of them: the half that is done first leaves the other's positions alone."""
    rng = np.random.default_rng(N + window)
    run(rng, [0, 3, 130, 260, 700], N, 2, G, D, 16, BF, parents=tree(rng, 5, N), window=window, slopes=slopes_of(2 * G))


@pytest.mark.parametrize("N,G", [(2, 4), (20, 4)])
@pytest.mark.parametrize("sm,cap", [(-0.3, 0.0), (-0.3, 4.0), (0.0, 0.0), (3.0, 0.0), (3.0, 20.0)])
def test_scales(N, G, sm, cap):
    run(np.random.default_rng(9), [3, 200], N, 1, G, 64, 16, BF, sm=sm, cap=cap)


@pytest.mark.parametrize("N,G", [(2, 4), (20, 4)])
@pytest.mark.parametrize("size,sm", [(2.0 ** 54, 2.0 ** -110), (2.0 ** 54, -2.0 ** -110), (2.0 ** 60, 2.0 ** -122), (2.0 ** 60, 0.0)])
def test_scales_as_small_as_their_products_are_large(N, G, size, sm):
    """Products of 2^120 at most 2^7 times in all: within fp32."""
    rng = np.random.default_rng(27)
    c = host_cache(rng, 20, 16, 1, 64, BF)
    c["k"] = c["k"] * size
    hq, gq = normal(rng, (2, N, G, 64), BF)
    run(rng, [3, 200], N, 1, G, 64, 16, BF, sm=sm, cache=c, pages=20, q=(hq * size, gq * size))


def test_negative_slopes_and_rising_maxima():
    """Scores that rise along the line, so that the running maximum does at every tile."""
    for N, G in ((2, 4), (40, 4)):
        run(np.random.default_rng(10), [900, 513], N, 1, G, 64, 16, BF, slopes=-np.array([0.1, 0.5, 0.0, 0.25]))
        run(np.random.default_rng(10), [900, 513], N, 1, G, 64, 16, F16, slopes=np.array([0.1, 0.5, 0.0, 2.0]))


# ------------------------------------------------------- pages, counts, trees that are bad

@pytest.mark.parametrize("N,G", [(5, 4), (40, 4)])
def test_counts_and_missing_pages(N, G):
    rng = np.random.default_rng(11)
    base = [100, 40, -1, 17, 0, 150]
    tab = table(rng, [250] * 6, 16, 120, width=16)
    tab[0, 2] = -1           # in the prefix
    tab[3, :] = 4000         # all of them
    n_nodes = [N, 0, N, N, 1, N + 1]
    r, want = run(rng, base, N, 2, G, 64, 16, BF, tab=tab, pages=120, n_nodes=n_nodes)
    assert r["status"].cpu().tolist() == [256, 0, 256, 256, 0, 256]
    assert (r["out"][1] == 0).all() and (r["out"][3] == 0).all() and (r["out"][4, 1:] == 0).all()


@pytest.mark.parametrize("N,G", [(5, 4), (40, 4)])
def test_a_table_that_is_too_short(N, G):
    rng = np.random.default_rng(12)
    r, _ = run(rng, [46, 47, 48, 60], N, 1, G, 64, 16, BF, tab=rng.permutation(12).reshape(4, 3), pages=12)
    assert (r["status"].cpu() == 256).all()


@pytest.mark.parametrize("N,G", [(5, 4), (70, 4)])
def test_pages_that_no_window_reaches_may_be_gone(N, G):
    rng = np.random.default_rng(13)
    tab = table(rng, [600, 600], 16, 90)
    tab[0, :(500 - 40 + 1) // 16] = -1
    tab[1, :(300 - 40 + 1) // 16] = 1 << 30
    r, _ = run(rng, [500, 300], N, 1, G, 64, 16, BF, tab=tab, pages=90, window=40)
    assert r["status"].cpu().tolist() == [0, 0]


@pytest.mark.parametrize("N,G", [(6, 4), (40, 4)])
def test_bad_parents(N, G):
    rng = np.random.default_rng(14)
    par = tree(rng, 4, N)
    par[0, 4], par[1, 3], par[2, 0] = 5, -1, 2
    par[3, 5] = -7
    r, _ = run(rng, [20, 130, 0, 64], N, 1, G, 64, 16, BF, parents=par)
    assert r["status"].cpu().tolist() == [2, 2, 2, 2]


@pytest.mark.parametrize("value", [-2, -32768, -32769, -40000, -65536, -(1 << 31), 1 << 16, (1 << 31) - 1])
@pytest.mark.parametrize("N,G,D", [(6, 4, 64), (40, 1, 64), (40, 4, 128), (150, 2, 64)])
def test_parents_far_out_of_range(value, N, G, D):
    """They end the path, at the root and inside a tree, whatever their low bits are."""
    rng = np.random.default_rng(23)
    par = tree(rng, 4, N)
    par[0, 0] = par[1, 3] = par[2, 0] = par[2, 4] = value
    r, _ = run(rng, [20, 130, 0, 64], N, 1, G, D, 16, BF, parents=par)
    assert r["status"].cpu().tolist() == [2, 2, 2, 0]


# ------------------------------------------------------- what must not be read

@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("N,G,window", [(6, 4, 0), (6, 4, 50), (40, 4, 0), (40, 4, 50), (1, 2, 7)])
def test_poison_in_slots_that_are_not_seen(dtype, N, G, window):
    rng = np.random.default_rng(15)
    base, P = [0, 37, 100, 250], 16
    par = tree(rng, 4, N)
    lens = [b + N for b in base]
    pages = sum(-(-n // P) for n in lens) + 2
    tab = table(rng, lens, P, pages)
    c = host_cache(rng, pages, P, 2, 64, dtype)
    for b, n in enumerate(lens):   # the last page behind the last row, and pages of no request
        c["k"][tab[b, (n - 1) // P], n % P or P:], c["v"][tab[b, (n - 1) // P], n % P or P:] = np.nan, np.inf
    loose = [p for p in range(pages) if p not in tab]
    c["k"][loose], c["v"][loose] = np.nan, np.nan
    r, want = run(rng, base, N, 2, G, 64, P, dtype, parents=par, window=window, tab=tab, pages=pages, cache=c)
    assert np.isfinite(want[0]).all()


@pytest.mark.parametrize("N,G", [(6, 4), (40, 4)])
def test_values_that_are_not_finite_reach_those_who_see_them(N, G):
    rng = np.random.default_rng(16)
    base, P = [37, 100], 16
    par = tree(rng, 2, N)
    tab = table(rng, [b + N for b in base], P, 30)
    c = host_cache(rng, 30, P, 1, 64, BF)
    at = lambda b, p: (tab[b, p // P], p % P, 0)  # noqa: E731
    c["v"][at(0, base[0] + 3)][5] = np.inf
    c["v"][at(0, base[0] + 4)][6] = np.nan
    c["v"][at(0, base[0] + 5)][7] = -np.inf
    c["v"][at(1, base[1] + 2)][[0, 63]] = np.inf
    c["v"][at(1, base[1] + 4)][[0, 62]] = -np.inf
    c["k"][at(1, base[1] + 5)][9] = np.nan
    r, want = run(rng, base, N, 1, G, 64, P, BF, parents=par, tab=tab, pages=30, cache=c)
    got = r["out"].double().cpu().numpy()
    odd = ~np.isfinite(want[0])
    assert odd.any() and np.array_equal(got[odd], want[0][odd], equal_nan=True)


@pytest.mark.parametrize("N,G", [(4, 4), (40, 4)])
def test_a_query_that_is_not_finite_spoils_its_row_alone(N, G):
    rng = np.random.default_rng(17)
    hq, gq = normal(rng, (1, N, G, 64), BF)
    hq[0, 2, 1, 5], gq[0, 2, 1, 5] = np.nan, float("nan")
    r, want = run(rng, [150], N, 1, G, 64, 16, BF, q=(hq, gq))
    got = torch.isnan(r["out"])[0].cpu()
    assert got[2, 1].all() and int(got.sum()) == 64


# ------------------------------------------------------- layouts, streams, graphs

@pytest.mark.parametrize("layout", ["hnd", "joint"])
@pytest.mark.parametrize("N,G", [(3, 4), (40, 4)])
def test_layouts(layout, N, G):
    run(np.random.default_rng(18), [9, 240], N, 3, G, 128, 16, BF, layout=layout)


def test_strided_queries():
    rng = np.random.default_rng(19)
    for N in (3, 40):
        hq, gq = normal(rng, (2, N, 4, 64), BF)
        joint = torch.cat([gq, torch.full_like(gq, float("nan"))], 2)[:, :, :4]
        odd = torch.empty((2, N, 4, 65), dtype=BF, device=DEV)[..., 1:]
        odd.copy_(gq)
        for t in (joint, odd, gq.transpose(0, 1).contiguous().transpose(0, 1)):
            run(np.random.default_rng(20), [50, 130], N, 1, 4, 64, 16, BF, q=(hq, t))


def big(B, N, H, G, D, P, L, dtype, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    W = -(-(L + N) // P)
    mk = lambda *s: torch.randn(s, generator=g, device=DEV).to(dtype)  # noqa: E731
    return (mk(B, N, H * G, D), sv.PagedCache(mk(B * W, P, H, D), mk(B * W, P, H, D)),
            torch.randperm(B * W, generator=g, device=DEV).view(B, W).int())


def in_64(q, cache, tab, base, window=0):
    """Chains in 64 bits with torch: (out, lse, sum p |v|, largest sum |q||k| sm, largest |score|, slots seen)."""
    B, N, Hq, D = q.shape
    H = cache.k.shape[2]
    res = [torch.empty((B, N, Hq, D), dtype=torch.float64) for _ in "oa"] + [torch.empty((B, N, Hq), dtype=torch.float64) for _ in "lszc"]
    for b in range(B):
        n = int(base[b]) + N
        k, v = (t[tab[b].long()].flatten(0, 1)[:n].double() for t in cache)
        far = (int(base[b]) + torch.arange(N, device=DEV))[:, None] - torch.arange(n, device=DEV)
        see = (far >= 0) & ((far < window) if window else (far >= 0))
        for h in range(Hq):
            kk, vv, qq = k[:, h * H // Hq], v[:, h * H // Hq], q[b, :, h].double()
            z = (qq @ kk.T * D ** -0.5).masked_fill(~see, -torch.inf)
            p = torch.softmax(z, -1)
            for t, x in zip(res, (p @ vv, p @ vv.abs(), torch.logsumexp(z, -1), (qq.abs() @ kk.abs().T * see).amax(-1) * D ** -0.5,
                                  z.masked_fill(~see, 0).abs().amax(-1), see.sum(-1).double())):
                t[b, :, h] = x.cpu()
    o, a, l, s, z, c = (t.numpy() for t in res)
    return o, l, a, s, z, c


@pytest.mark.parametrize("B,N,H,G,D,L,window,dtype", [
    (1, 1, 1, 4, 128, 70001, 0, BF), (3, 2, 2, 8, 64, 33333, 0, F16), (2, 6, 1, 4, 128, 50000, 4097, BF),
    (1, 64, 1, 4, 128, 20000, 0, BF), (2, 700, 2, 4, 128, 999, 0, BF), (1, 1500, 1, 8, 64, 0, 0, F16), (1, 1200, 1, 4, 64, 3000, 513, BF)])
def test_long_lines(B, N, H, G, D, L, window, dtype):
    q, cache, tab = big(B, N, H, G, D, 16, L, dtype, N + L)
    base = [max(0, L - 1000 * b) for b in range(B)]
    r = sv.spec_attention(q, cache, tab, i32(base), window=window)
    check_attention(r, in_64(q, cache, tab, base, window), dtype, N * G)


def test_offsets_past_32_bits():
    """A cache of more than 2^32 bytes whose last pages are read."""
    pages = (1 << 32) // (128 * 2 * 128 * 2) + 8
    k = torch.zeros((pages, 128, 2, 128), dtype=BF, device=DEV)
    v = torch.zeros_like(k)
    q, small, tab = big(1, 40, 2, 4, 128, 128, 300, BF, 3)
    n = small.k.shape[0]
    k[-n:], v[-n:] = small.k, small.v
    for rows in (2, 40):
        a = sv.spec_attention(q[:, :rows], small, tab, i32([300]))
        b = sv.spec_attention(q[:, :rows], sv.PagedCache(k, v), tab + (pages - n), i32([300]))
        assert torch.equal(a["out"], b["out"]) and torch.equal(a["lse"], b["lse"])


def test_same_again_other_streams_and_graphs():
    """Bit for bit the same on another stream, with buffers given, and from two graphs whose replays interleave."""
    base = i32([700, 90, 5000])
    for N, G in ((3, 4), (40, 4)):
        q, cache, tab = big(3, N, 2, G, 128, 16, 5000, BF, 1)
        first = sv.spec_attention(q, cache, tab, base)
        size = sv.load_library().spec_attention_workspace_size(3, N, 2 * G, 2, 128)
        out = {n: torch.empty_like(first[n]) for n in first}
        ws = torch.empty(size, dtype=torch.uint8, device=DEV)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            sv.spec_attention(q, cache, tab, base, workspace=ws, out=out)
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(first[n], out[n]) for n in first)
        graphs = []
        for w in (0, 100):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                graphs.append((g, sv.spec_attention(q, cache, tab, base, window=w), w))
        sv.spec_attention(q, cache, tab, base)   # a call between, on the kept workspace
        sides = [torch.cuda.Stream() for _ in graphs]
        for s, (g, _, _) in zip(sides, graphs):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for _, got, w in graphs:
            want = sv.spec_attention(q, cache, tab, base, window=w)
            assert all(torch.equal(got[n], want[n]) for n in got)


def test_requests_that_share_pages_and_many_of_them():
    q, cache, _ = big(300, 1, 1, 4, 64, 16, 0, BF, 2)
    tab = torch.arange(4, dtype=torch.int32, device=DEV).repeat(300, 1)
    base = [(i * 7) % 63 for i in range(300)]
    r = sv.spec_attention(q, cache, tab, i32(base))
    check_attention(r, in_64(q, cache, tab, base), BF, 4)


def test_no_requests():
    c = sv.paged_cache(2, 2, 16, 64)
    e = torch.empty((0, 3, 4, 64), dtype=BF, device=DEV)
    assert sv.spec_attention(e, c, i32(np.zeros((0, 2))), i32([]))["out"].shape == (0, 3, 4, 64)


# ------------------------------------------------------- many pieces, refusals from Python

@pytest.mark.parametrize("B,N,H,G,D,L,dtype", [
    (40, 75, 3, 4, 128, 300, BF), (30, 150, 2, 2, 64, 500, F16), (70, 12, 4, 4, 64, 700, BF), (90, 9, 3, 5, 128, 260, F16),
    (200, 1, 8, 4, 128, 200, BF), (150, 5, 8, 5, 64, 300, F16), (3, 1301, 2, 7, 64, 100, BF)])
def test_many_pieces(B, N, H, G, D, L, dtype):
    """Every CTA has many items, of blocks with one half and with two, some of them shared with its neighbours."""
    q, cache, tab = big(B, N, H, G, D, 16, L, dtype, N + L)
    base = [(L * (7 * b % B)) // B for b in range(B)]
    r = sv.spec_attention(q, cache, tab, i32(base))
    assert int(r["status"].max()) == 0
    check_attention(r, in_64(q, cache, tab, base), dtype, N * G)


@pytest.mark.parametrize("N,D", [(9, 128), (9, 64), (2, 128)])
def test_more_requests_than_threads(N, D):
    q, cache, _ = big(900, N, 1, 4, D, 16, 0, BF, 4)
    tab = torch.arange(8, dtype=torch.int32, device=DEV).repeat(900, 1)
    base = [(i * 37) % 110 for i in range(900)]
    r = sv.spec_attention(q, cache, tab, i32(base))
    assert int(r["status"].max()) == 0
    check_attention(r, in_64(q, cache, tab, base), BF, N * 4)


@pytest.mark.parametrize("D,G", [(64, 2), (128, 1)])
def test_more_blocks_than_threads(D, G):
    """A prompt of 150,000 rows in a window of 100; every 997th row and the last ones against 64 bits."""
    N, w = 150_000, 100
    q, cache, tab = big(1, N, 1, G, D, 64, 0, BF, 5)
    r = sv.spec_attention(q, cache, tab, i32([0]), window=w)
    assert int(r["status"].max()) == 0
    rows = torch.tensor([*range(0, N, 997), *range(N - 40, N)], device=DEV)
    at = rows[:, None] - torch.arange(w, device=DEV)
    see = (at >= 0)[:, None]
    k, v = (t[tab[0].long()].flatten(0, 1)[at.clamp(min=0)][:, :, 0].double() for t in cache)   # [rows, w, D]
    qq = q[0, rows].double()
    z = torch.einsum("rgd,rwd->rgw", qq, k).mul(D ** -0.5).masked_fill(~see, -torch.inf)
    p = torch.softmax(z, -1)
    want = (p @ v, torch.logsumexp(z, -1), p @ v.abs(), torch.einsum("rgd,rwd->rgw", qq.abs(), k.abs()).amax(-1) * D ** -0.5,
            z.masked_fill(~see, 0).abs().amax(-1), see.sum(-1).double().expand(-1, G))
    check_attention(dict(out=r["out"][:, rows], lse=r["lse"][:, rows]), [t.cpu().numpy()[None] for t in want], BF, N * G)


@pytest.mark.parametrize("D", [64, 128])
def test_blocks_of_two_halves_and_of_one_by_turns(D):
    """Pieces of two halves go over to pieces of one and back in every CTA, again and again the same bits."""
    q, cache, tab = big(40, 70, 2, 4, D, 16, 1500, F16, 25)
    base = i32([(1500 * (7 * b % 40)) // 40 for b in range(40)])
    first = sv.spec_attention(q, cache, tab, base)
    assert int(first["status"].max()) == 0
    check_attention(first, in_64(q, cache, tab, base.tolist()), F16, 280)
    for _ in range(20):
        r = sv.spec_attention(q, cache, tab, base)
        assert all(torch.equal(r[n], first[n]) for n in r)


@pytest.mark.parametrize("D,dtype", [(128, BF), (64, F16)])
def test_a_half_without_rows_waits_through_long_pieces(D, dtype):
    """65 rows of 4 heads after 190 million tokens: a block of 256 rows and one of 4, of which one CTA has some 30,000 tiles
    (longer than any wait's limit) before a block of 256 of the next request. The prefix goes round 64 pages, so it is one
    round with every weight counted `turns` times."""
    N, G, turns = 65, 4, (23400, 22900)
    g = torch.Generator(device=DEV).manual_seed(24)
    mk = lambda *s: torch.randn(s, generator=g, device=DEV).to(dtype)  # noqa: E731
    q, cache = mk(2, N, G, D), sv.PagedCache(mk(66, 128, 1, D), mk(66, 128, 1, D))
    tab = (torch.arange(64 * turns[0] + 1, device=DEV, dtype=torch.int32) % 64).repeat(2, 1)
    for b, n in enumerate(turns):
        tab[b, 64 * n] = 64 + b
    r = sv.spec_attention(q, cache, tab, i32([8192 * n for n in turns]))
    assert r["status"].cpu().tolist() == [0, 0]
    for b, n in enumerate(turns):
        k, v = (torch.cat([t[:64].flatten(0, 1), t[64 + b, :N]])[:, 0].double() for t in cache)
        z = torch.einsum("ngd,sd->ngs", q[b].double(), k) * D ** -0.5
        z[..., :8192] += np.log(n)
        z.masked_fill_((torch.arange(8192 + N, device=DEV) > 8192 + torch.arange(N, device=DEV)[:, None])[:, None], -torch.inf)
        p = torch.softmax(z, -1)
        # A CTA sums up to 40,000 tiles, eight products of 16 slots a tile, each sum off by a step of fp32 (2^-23); besides
        # that the weights' and the output's rounding, and scores off by 2^-16 of a sum of at most 64 or so.
        off = 8 * 40000 * 2.0 ** -23 + 2.0 ** -10
        assert ((r["lse"][b] - torch.logsumexp(z, -1)).abs() < off).all()
        assert ((r["out"][b].double() - p @ v).abs() < (2 * off + 2.0 ** -7) * (p @ v.abs())).all()


@pytest.mark.parametrize("N,G", [(2, 4), (12, 4), (70, 4)])
def test_nan_keys_under_a_cap(N, G):
    rng = np.random.default_rng(21)
    c = host_cache(rng, 30, 16, 1, 64, BF)
    tab = table(rng, [200 + N], 16, 30)
    c["k"][tab[0, 3], 5, 0, 9] = np.nan      # a slot that every row sees
    r, want = run(rng, [200], N, 1, G, 64, 16, BF, cap=20.0, tab=tab, pages=30, cache=c)
    assert torch.isnan(r["out"]).all() and torch.isnan(r["lse"]).all()


@pytest.mark.parametrize("N,G,tree_rows", [(6, 4, False), (36, 1, False), (10, 4, True), (130, 2, False)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("low", [0, 1, 2])
@pytest.mark.parametrize("what", ["k nan", "k all nan", "v nan", "v inf", "v last inf"])
def test_what_is_not_finite_far_below_the_maximum(N, G, tree_rows, D, low, what):
    """Scores of one tile are 200 or more below the others', so its weights are zero to fp32; what is not finite there still
    shows. 300 requests with the same rows, so that CTAs have all tiles of an item and parts of one."""
    rng = np.random.default_rng(26)
    base = 256 + 40
    tab = table(rng, [base + N], 16, 30)
    c = host_cache(rng, 30, 16, 1, D, BF)
    hq, gq = normal(rng, (1, N, G, D), BF)
    hq[..., 0], gq[..., 0] = 8.0, 8.0
    spots = [(tab[0, p // 16], p % 16) for p in range(base)]
    for p, at in enumerate(spots):
        c["k"][at][0, 0] = 0.0 if p // 128 == low else 300.0
    at = [spots[p] for p in range(base) if p // 128 == low]
    if what == "k nan":
        c["k"][at[3]][0, 9] = np.nan
    elif what == "k all nan":
        for x in at:
            c["k"][x][0, 9] = np.nan
    elif what == "v nan":
        c["v"][at[3]][0, 9] = np.nan
    else:
        c["v"][at[-1 if "last" in what else 3]][0, 9] = np.inf
    parents = tree(rng, 1, N) if tree_rows else None
    c = {n: torch.from_numpy(x).to(BF).double().numpy() for n, x in c.items()}
    want = K.attention(hq, c, tab, [base], parents, None, D ** -0.5)
    many = lambda x: i32(x).expand(300, -1).contiguous()  # noqa: E731
    r = sv.spec_attention(gq.expand(300, -1, -1, -1), to_gpu(c, BF), many(tab), i32([base] * 300),
                          parents=many(parents) if tree_rows else None)
    check_attention(r, [np.repeat(x, 300, 0) for x in want], BF, N * G)
    lost = np.isnan(want[1]) if "k" in what else ~np.isfinite(want[0][..., 9])
    assert lost.all()


@pytest.mark.parametrize("N,G", [(2, 4), (12, 4), (70, 4)])
@pytest.mark.parametrize("cap", [1.0, 30.0])
def test_scores_far_past_the_cap(N, G, cap):
    run(np.random.default_rng(22), [150, 3], N, 1, G, 64, 16, BF, cap=cap, q_std=300.0)


@pytest.mark.parametrize("N,G,tree_rows", [(2, 4, False), (20, 1, True), (12, 4, True), (70, 4, False)])
@pytest.mark.parametrize("cap,q_std", [(129.0, 2.0), (1e4, 2.0), (1e6, 8.0), (1e30, 2.0), (2e38, 2.0), (200.0, 300.0), (1000.0, 300.0)])
def test_caps_that_are_large(N, G, tree_rows, cap, q_std):
    """Below a quarter of the cap a score is off by 2^-21 of itself, above by 2^-20 of the cap, so 2^-18 of itself: a part of
    the 2^-16 of its |q||k| that its product may be off by."""
    rng, base, D = np.random.default_rng(28), [150, 3], 64
    tab = table(rng, [b + N for b in base], 16, 20)
    c = host_cache(rng, 20, 16, 1, D, F16)
    hq, gq = normal(rng, (2, N, G, D), F16, q_std)
    par = tree(rng, 2, N) if tree_rows else None
    r = sv.spec_attention(gq, to_gpu(c, F16), i32(tab), i32(base), parents=i32(par) if tree_rows else None, softcap=cap)
    check_attention(r, K.attention(hq, c, tab, base, par, sm=D ** -0.5, cap=cap), F16, N * G)


# ------------------------------------------------------- 128-wide heads, deep trees, prompts with all of it

@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("N,G,window", [(6, 4, 0), (36, 1, 50), (70, 4, 0), (70, 4, 50), (5, 5, 7)])
def test_poison_beside_wide_heads(dtype, N, G, window):
    rng = np.random.default_rng(29)
    base, P, D = [0, 37, 100, 250], 64, 128
    par, lens = tree(rng, 4, N), [b + N for b in base]
    pages = sum(-(-n // P) for n in lens) + 2
    tab = table(rng, lens, P, pages)
    c = host_cache(rng, pages, P, 2, D, dtype)
    for b, n in enumerate(lens):
        if n % P:
            c["k"][tab[b, n // P], n % P:], c["v"][tab[b, n // P], n % P:] = np.nan, np.inf
    loose = [p for p in range(pages) if p not in tab]
    c["k"][loose], c["v"][loose] = np.nan, np.nan
    r, want = run(rng, base, N, 2, G, D, P, dtype, parents=par, window=window, tab=tab, pages=pages, cache=c)
    assert np.isfinite(want[0]).all()


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("N,G", [(6, 4), (36, 1), (70, 4)])
def test_values_of_wide_heads_that_are_not_finite(dtype, N, G):
    """In the prefix, in whole tiles and ragged ones, and in nodes that some rows see and others do not."""
    rng = np.random.default_rng(30)
    base, P, D = [200, 37], 64, 128
    par = tree(rng, 2, N)
    tab = table(rng, [b + N for b in base], P, 12)
    c = host_cache(rng, 12, P, 1, D, dtype)
    at = lambda b, p: (tab[b, p // P], p % P, 0)  # noqa: E731
    for slot, d, x in ((3, 5, np.inf), (130, 64, np.nan), (199, 127, -np.inf), (202, 31, np.inf), (205, 96, np.nan)):
        c["v"][at(0, slot)][d] = x
    for slot, d, x in ((39, 0, np.inf), (39, 127, -np.inf), (41, 0, -np.inf), (42, 95, np.nan)):
        c["v"][at(1, slot)][d] = x
    r, want = run(rng, base, N, 1, G, D, P, dtype, parents=par, tab=tab, pages=12, cache=c)
    got, odd = r["out"].double().cpu().numpy(), ~np.isfinite(want[0])
    # in a tile that every row sees whole an infinity may also be NaN (the second of a weight's two terms has either sign)
    whole = np.zeros_like(odd)
    whole[0, ..., 5] = True
    assert odd.any() and np.array_equal(got[odd & ~whole], want[0][odd & ~whole], equal_nan=True)


@pytest.mark.parametrize("N,G,D,depth", [(300, 1, 64, 200), (1024, 1, 128, 1024), (90, 2, 64, 60), (31, 1, 64, 31)])
def test_deep_trees(N, G, D, depth):
    rng = np.random.default_rng(31)
    par = np.array([[-1] + [n - 1 if n < depth else int(rng.integers(n)) for n in range(1, N)]])
    run(rng, [70], N, 1, G, D, 16, F16, parents=par, window=0 if N < 100 else 150, slopes=slopes_of(G) if N == 300 else None)


def in_64_scored(q, cache, tab, base, window=0, cap=0.0, slopes=None):
    """in_64 for capped and biased scores."""
    B, N, Hq, D = q.shape
    H, o = cache.k.shape[2], []
    for b in range(B):
        n = base[b] + N
        k, v = (t[tab[b].long()].flatten(0, 1)[:n].double().repeat_interleave(Hq // H, 1) for t in cache)
        far = ((base[b] + torch.arange(N, device=DEV))[:, None] - torch.arange(n, device=DEV))[None]
        see = (far >= 0) & ((far < window) if window else (far >= 0))
        z = torch.einsum("nhd,shd->hns", q[b].double(), k) * D ** -0.5
        z = cap * torch.tanh(z / cap) if cap else z
        z = z if slopes is None else z - torch.tensor(slopes, device=DEV)[:, None, None] * far
        hid = z.masked_fill(~see, -torch.inf)
        p = torch.softmax(hid, -1)
        o.append([torch.einsum("hns,shd->nhd", p, v), torch.logsumexp(hid, -1).T, torch.einsum("hns,shd->nhd", p, v.abs()),
                  (torch.einsum("nhd,shd->hns", q[b].double().abs(), k.abs()) * see).amax(-1).T * D ** -0.5,
                  z.masked_fill(~see, 0).abs().amax(-1).T, see.sum(-1).double().expand(Hq, -1).T])
    return [torch.stack(x).cpu().numpy() for x in zip(*o)]


@pytest.mark.parametrize("D,G,dtype", [(128, 4, BF), (64, 8, F16), (128, 1, F16), (64, 2, BF)])
@pytest.mark.parametrize("cap,window,bias", [(50.0, 0, False), (30.0, 300, False), (0.0, 129, True), (50.0, 512, True), (1000.0, 0, False)])
def test_prompts_with_caps_windows_and_biases(D, G, dtype, cap, window, bias):
    N = 1001 if G < 8 else 600
    q, cache, tab = big(2, N, 2, G, D, 32, 700, dtype, 32)
    q, base, slopes = (q * 4).to(dtype), [700, 33], slopes_of(2 * G) if bias else None
    r = sv.spec_attention(q, cache, tab, i32(base), softcap=cap, window=window,
                          slopes=None if slopes is None else torch.tensor(slopes, dtype=torch.float32, device=DEV))
    assert int(r["status"].max()) == 0
    check_attention(r, in_64_scored(q, cache, tab, base, window, cap, slopes), dtype, N * G, cap if cap <= 128 else 0.0)


def test_python_refusals():
    E = sv.SpecVerifyError
    c = sv.paged_cache(4, 2, 16, 64)
    q = torch.zeros((2, 3, 4, 64), dtype=BF, device=DEV)
    tab, base = i32([[0, 1], [2, 3]]), i32([0, 5])
    ok = sv.spec_attention(q, c, tab, base)
    for bad in (dict(q=q[..., :32]), dict(q=q[:, :, :3]), dict(q=q.half()), dict(q=q.float()), dict(q=q[0]), dict(q=q.cpu()),
                dict(page_table=tab[:1]), dict(seq_base=base[:1]), dict(parents=i32([[0]])), dict(n_nodes=i32([1])), dict(window=-1),
                dict(softcap=-1.0), dict(softcap=float("nan")), dict(slopes=torch.zeros(3, device=DEV)), dict(slopes=torch.zeros(4)),
                dict(workspace=torch.zeros(8, device=DEV)), dict(out=[]), dict(out={}), dict(cache=(c.k,)), dict(cache=(c.k, c.v[:2])),
                dict(cache=(c.k, c.v.half())), dict(cache=(c.k.float(), c.v.float())), dict(cache=(c.k[:, :8], c.v[:, :8])),
                dict(cache=(c.k[..., ::2], c.v[..., ::2])), dict(cache=tuple(t.transpose(1, 3) for t in c)),
                dict(cache=tuple(t.expand(4, 16, 2, 64)[:, :, :1].expand(4, 16, 2, 64) for t in c))):
        a = dict(q=q, cache=c, page_table=tab, seq_base=base)
        a.update(bad)
        with pytest.raises(E):
            sv.spec_attention(**a)
    k = torch.zeros((2, 3, 2, 64), dtype=BF, device=DEV)
    f = torch.ones(32, device=DEV)
    for bad in (dict(k_new=k[:, :, :1]), dict(v_new=k[:1]), dict(k_new=k.half()), dict(inv_freq=f.double()), dict(inv_freq=f[:31]),
                dict(inv_freq=f.repeat(2)), dict(inv_freq=f.cpu()), dict(q=q[:, :2]), dict(q=q.half()), dict(parents=i32([[0]])),
                dict(n_nodes=i32([1])), dict(page_table=tab[0]), dict(out=dict(out_len=base, status=torch.empty_like(base)))):
        a = dict(cache=c, k_new=k, v_new=k, page_table=tab, seq_base=base, inv_freq=f)
        a.update(bad)
        with pytest.raises(E):
            sv.spec_kv_append_rope(**a)
    with pytest.raises(E):
        sv.spec_attention(torch.zeros((1, 1025, 2, 64), dtype=BF, device=DEV), c, tab[:1], base[:1], parents=torch.zeros((1, 1025), dtype=torch.int32, device=DEV))
    assert torch.equal(sv.spec_attention(q, c, tab, base)["out"], ok["out"])
