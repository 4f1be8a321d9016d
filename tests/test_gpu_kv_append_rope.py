"""Appending to the 16-bit paged cache with the rotation on the way, against the oracle."""

import numpy as np
import pytest
import torch

import speculative_decoding_verification_72_gb300 as sv
from oracle import kv_paged as K
from paged_utils import DEV, U, host_cache, i32, inv_freq, normal, table, to_gpu, to_host, tree

pytestmark = pytest.mark.gpu


def same(got, want, x_max, dtype):
    """One rounding of the type on top of fp32: three roundings of numbers up to the pair's length and an angle that is off
    by 2^-24 of a turn."""
    fine = U[dtype] * np.abs(want) * 1.001 + x_max * (2 * np.pi * 2.0 ** -24 + 6 * 2.0 ** -24) + 2.0 ** -25
    assert (np.abs(got - want) <= fine).all(), (np.abs(got - want) - fine).max()


def run(rng, base, N, H, Hq, D, P, dtype, rot=None, interleaved=False, parents=None, n_nodes=None, layout="nhd", tab=None, pages=None,
        q_given=True, split=False):
    B, rot = len(base), rot or D
    lens = [b + N for b in base]
    pages = pages or sum(-(-n // P) for n in lens) + 2
    tab = table(rng, lens, P, pages) if tab is None else tab
    c = host_cache(rng, pages, P, H, D, dtype)
    (hk, k), (hv, v), (hq, q) = (normal(rng, (B, N, h, D), dtype) for h in (H, H, Hq))
    if split:   # as a fused projection leaves them: slices of one row
        joint = torch.cat([q, k, v], 2)
        q, k, v = joint.split([Hq, H, H], 2)
    f = inv_freq(rot)
    cache = to_gpu(c, dtype, layout)
    r = sv.spec_kv_append_rope(cache, k, v, i32(tab), i32(base), torch.from_numpy(f).to(DEV), q=q if q_given else None,
                               parents=None if parents is None else i32(parents), n_nodes=None if n_nodes is None else i32(n_nodes),
                               interleaved=interleaved)
    want, n, st, wq = K.append_rope(c, hk, hv, tab, base, f, hq, parents, n_nodes, interleaved)
    got = to_host(cache)
    new = ~np.all(want["k"] == c["k"], -1)
    assert np.array_equal(got["k"][~new], c["k"][~new])   # what no row lands on
    same(got["k"], want["k"], np.abs(hk).max() * 1.5, dtype)
    assert np.array_equal(got["v"], want["v"])
    assert r["out_len"].cpu().tolist() == n.tolist() and r["status"].cpu().tolist() == st.tolist()
    if q_given:
        same(r["q"].double().cpu().numpy(), wq, np.abs(hq).max() * 1.5, dtype)
    else:
        assert "q" not in r
    return r


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D,P,H,Hq", [(128, 16, 2, 8), (64, 32, 1, 7), (64, 128, 3, 3), (128, 64, 8, 32)])
@pytest.mark.parametrize("N,base", [(1, [0]), (1, [5, 16, 127]), (6, [0, 15, 100, 61]), (70, [3, 64])])
def test_chains(dtype, D, P, H, Hq, N, base):
    run(np.random.default_rng(N + D), base, N, H, Hq, D, P, dtype)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot", [(128, 16), (128, 112), (64, 48), (64, 64)])
def test_a_part_of_the_head(interleaved, D, rot):
    run(np.random.default_rng(rot), [9, 40], 5, 2, 4, D, 16, torch.bfloat16, rot=rot, interleaved=interleaved)


@pytest.mark.parametrize("N", [2, 33, 64])
def test_trees(N):
    rng = np.random.default_rng(N)
    run(rng, [17, 0, 300], N, 2, 8, 64, 16, torch.float16, parents=tree(rng, 3, N), interleaved=True)


@pytest.mark.parametrize("layout", ["hnd", "joint"])
def test_layouts_and_slices(layout):
    run(np.random.default_rng(1), [9, 40], 20, 2, 4, 128, 16, torch.bfloat16, layout=layout, split=True)


def test_long_prompt_without_queries():
    run(np.random.default_rng(2), [7], 1000, 1, 1, 64, 16, torch.bfloat16, q_given=False)


def test_ragged_counts_and_rows_behind_them():
    rng = np.random.default_rng(3)
    r = run(rng, [10, 20, 30, 40], 9, 2, 4, 64, 16, torch.bfloat16, n_nodes=[9, 0, 1, 5])
    assert (r["q"][1] == 0).all() and (r["q"][3, 5:] == 0).all() and (r["q"][3, :5] != 0).any()


def test_bad_pages_counts_parents():
    rng = np.random.default_rng(4)
    tab = np.array([[0, 1, 2], [3, 99, 4], [5, -1, 6], [7, 8, 9], [10, 11, 12], [13, 14, 15], [16, 17, 18]])
    par = np.tile(np.arange(-1, 7), (7, 1))
    par[5, 3] = 6      # no earlier node
    par[6, 0] = 0
    r = run(rng, [4, 14, 30, 44, -3, 10, 10], 8, 2, 4, 64, 16, torch.bfloat16, tab=tab, pages=20, parents=par,
            n_nodes=[9, 8, 8, 8, 8, 8, 8])
    assert r["status"].cpu().tolist() == [256, 256, 256, 256, 256, 2, 2]
    assert (r["q"][4] == 0).all()


@pytest.mark.parametrize("value", [-2, -32768, -40000, -65536, -(1 << 31), 1 << 16, (1 << 31) - 1])
def test_parents_far_out_of_range(value):
    rng = np.random.default_rng(8)
    par = tree(rng, 3, 40)
    par[0, 0] = par[1, 3] = value
    r = run(rng, [20, 130, 0], 40, 2, 4, 64, 16, torch.bfloat16, parents=par)
    assert r["status"].cpu().tolist() == [2, 2, 0]


def test_a_chain_given_as_a_tree():
    """The deepest tree that is taken: bit for bit a chain's rows."""
    rng = np.random.default_rng(10)
    N, H, D, P = 1024, 2, 64, 64
    (_, k), (_, v), (_, q) = (normal(rng, (2, N, h, D), torch.bfloat16) for h in (H, H, 4))
    base, tab, f = i32([40, 7]), i32(table(rng, [40 + N, 7 + N], P, 40)), torch.from_numpy(inv_freq(D)).to(DEV)
    one, two = sv.paged_cache(40, H, P, D), sv.paged_cache(40, H, P, D)
    par = i32(np.tile(np.arange(-1, N - 1), (2, 1)))
    a = sv.spec_kv_append_rope(one, k, v, tab, base, f, q=q, parents=par)
    b = sv.spec_kv_append_rope(two, k, v, tab, base, f, q=q)
    assert all(torch.equal(a[n], b[n]) for n in b) and torch.equal(one.k, two.k) and torch.equal(one.v, two.v)


def test_far_positions():
    """Angles of thousands of turns: positions near 2^20 and 2^24 in a table whose other pages are missing."""
    for base in (1 << 20, (1 << 24) - 40):
        rng = np.random.default_rng(5)
        W = base // 128 + 1
        tab = np.full((1, W), -1)
        tab[0, -1] = 2
        run(rng, [base], 16, 1, 2, 128, 128, torch.float16, tab=tab, pages=3)


def test_positions_near_the_end_of_32_bits():
    """The last slots of the longest table; angles of 2^28 turns, right to 2^-17 of one."""
    W, rng = (2 ** 31 - 256) // 128, np.random.default_rng(9)
    base, f = W * 128 - 40, inv_freq(128)
    tab = torch.full((1, W), -1, dtype=torch.int32, device=DEV)
    tab[0, -1] = 2
    c = sv.paged_cache(3, 1, 128, 128, torch.float16)
    (hk, k), (hq, q) = (normal(rng, (1, 16, h, 128), torch.float16) for h in (1, 2))
    r = sv.spec_kv_append_rope(c, k, k, tab, i32([base]), torch.from_numpy(f).to(DEV), q=q)
    assert r["status"].item() == 0 and r["out_len"].item() == base + 16
    for got, x in ((c.k[2, 88:104], hk), (r["q"][0], hq)):
        want = K.turn(x[0], base + np.arange(16), f)
        bound = U[torch.float16] * np.abs(want) * 1.001 + np.abs(x).max() * 1.5 * (2 * np.pi * 2.0 ** -17 + 6 * 2.0 ** -24) + 2.0 ** -25
        assert (np.abs(got.double().cpu().numpy() - want) <= bound).all()


def test_offsets_past_32_bits():
    """A cache of more than 2^32 bytes; the rows land on its last page."""
    pages = (1 << 32) // (128 * 2 * 128 * 2) + 3
    k = torch.zeros((pages, 128, 2, 128), dtype=torch.bfloat16, device=DEV)
    v = torch.zeros_like(k)
    rng = np.random.default_rng(6)
    (hk, kn), (hv, vn) = (normal(rng, (1, 3, 2, 128), torch.bfloat16) for _ in range(2))
    f = inv_freq(128)
    sv.spec_kv_append_rope(sv.PagedCache(k, v), kn, vn, i32([[pages - 1]]), i32([100]), torch.from_numpy(f).to(DEV))
    same(k[-1, 100:103].double().cpu().numpy(), K.turn(hk[0], [100, 101, 102], f), 6.0, torch.bfloat16)
    assert torch.equal(v[-1, 100:103], vn[0]) and int((k[:-1].view(torch.int16) != 0).sum()) == 0


def test_queries_in_place_out_and_capture():
    rng = np.random.default_rng(7)
    B, N, H, Hq, D, P = 3, 6, 2, 8, 128, 16
    base, f = [5, 30, 0], torch.from_numpy(inv_freq(128)).to(DEV)
    tab = i32(table(rng, [b + N for b in base], P, 9))
    k, v, q = (normal(rng, (B, N, h, D), torch.bfloat16)[1] for h in (H, H, Hq))
    want, cache = sv.paged_cache(9, H, P, D), sv.paged_cache(9, H, P, D)
    r = sv.spec_kv_append_rope(want, k, v, tab, i32(base), f, q=q)
    at = i32(base)
    out = dict(q=q.clone(), out_len=torch.empty_like(at), status=torch.empty_like(at))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        sv.spec_kv_append_rope(cache, k, v, tab, at, f, q=out["q"], out=out)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out["q"], r["q"]) and torch.equal(cache.k, want.k) and torch.equal(cache.v, want.v)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c = sv.spec_kv_append_rope(cache, k, v, tab, at, f, q=q)
    cache.k.zero_()
    k.mul_(2)   # the replay reads what is there then
    g.replay()
    torch.cuda.synchronize()
    sv.spec_kv_append_rope(want, k, v, tab, at, f)
    assert torch.equal(cache.k, want.k) and torch.equal(c["q"], r["q"]) and c["out_len"].tolist() == [11, 36, 6]


def test_no_requests():
    c = sv.paged_cache(2, 2, 16, 64)
    e = torch.empty((0, 3, 2, 64), dtype=torch.bfloat16, device=DEV)
    r = sv.spec_kv_append_rope(c, e, e, i32(np.zeros((0, 2))), i32([]), torch.ones(32, device=DEV), q=e)
    assert r["out_len"].shape == (0,) and r["q"].shape == (0, 3, 2, 64)
