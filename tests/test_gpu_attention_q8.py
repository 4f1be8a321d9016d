"""GPU parity of attention over the 8-bit cache, and of accumulated attention weight, against oracle/kv_q8.py."""

import numpy as np
import pytest
import torch

import speculative_decoding_verification_72_gb300 as sv
from speculative_decoding_verification_72_gb300 import workloads as W
from oracle import kv_q8 as K
from q8_utils import DEV, check_attention, host_cache, i32, rows, table, to_gpu

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    sv.load_library()


def trees(rng, B, N, topk=4, depth=5):
    return np.stack([W.tree_shape(rng, depth, topk, N) for _ in range(B)])


def problem(seed, base, N, H, G, D, P, dtype, pow2=True, q_std=2.0):
    rng = np.random.default_rng(seed)
    lens = [b + N for b in base]
    pages = sum(-(-n // P) for n in lens) + 3
    c = host_cache(rng, pages, H, P, D, pow2)
    t = table(rng, lens, P, pages)
    q, q64 = rows(rng, (len(base), N, H * G, D), dtype, q_std)
    return rng, c, t, q, q64


CASES = [  # base lengths, N, H, G, D, P, dtype, tree
    ([0], 1, 1, 1, 64, 16, BF, False),                              # one position
    ([0, 1, 15, 16, 17], 1, 2, 4, 128, 16, BF, False),              # around a page
    ([63, 64, 65, 127, 200], 3, 2, 5, 128, 32, HF, False),          # around a tile, an odd group
    ([100, 0, 31], 6, 2, 4, 128, 16, BF, False),                    # 24 rows
    ([700, 5, 300], 5, 1, 8, 64, 64, HF, False),
    ([1500], 1, 2, 1, 128, 128, BF, False),                         # many pieces of one item
    ([130, 77], 64, 2, 4, 128, 16, BF, True),                       # 256 rows, trees
    ([300, 0], 33, 2, 3, 64, 32, HF, True),                         # a tree that starts the cache
    ([90, 1000], 40, 1, 7, 128, 64, BF, True),
    ([10], 130, 1, 1, 64, 16, HF, False),                           # more nodes than three mask words
    ([60], 17, 1, 16, 128, 128, BF, True),
]


@pytest.mark.parametrize("base,N,H,G,D,P,dtype,tree", CASES)
def test_attention(base, N, H, G, D, P, dtype, tree):
    rng, c, t, q, q64 = problem(len(base) * 31 + N, base, N, H, G, D, P, dtype)
    par = trees(rng, len(base), N) if tree else None
    r = sv.spec_attention_q8(q, to_gpu(c), i32(t), i32(base), parents=None if par is None else i32(par))
    check_attention(r, K.attention(q64, c, t, base, par, sm=D ** -0.5), dtype)
    assert r["status"].tolist() == [0] * len(base)


@pytest.mark.parametrize("N,G,dtype", [(2, 4, BF), (4, 8, HF), (20, 8, BF)])
def test_any_scales_and_sharp_scores(N, G, dtype):
    base = [400, 90]
    rng, c, t, q, q64 = problem(5, base, N, 2, G, 128, 16, dtype, pow2=False, q_std=20.0)
    c["vs"][::2] *= 1e-3        # pages of very different magnitudes
    c["vs"][1] = 0.0
    c["vs"], c["ks"] = c["vs"].astype(np.float32).astype(np.float64), c["ks"].astype(np.float32).astype(np.float64)
    r = sv.spec_attention_q8(q, to_gpu(c), i32(t), i32(base), sm_scale=0.05)
    check_attention(r, K.attention(q64, c, t, base, sm=np.float64(np.float32(0.05))), dtype)


@pytest.mark.parametrize("N,G", [(6, 4), (40, 4)])
def test_rows_that_see_nothing(N, G):
    base = [40, 0, 7]
    rng, c, t, q, q64 = problem(6, base, N, 2, G, 64, 16, BF)
    nn = [N, 0, 3]
    r = sv.spec_attention_q8(q, to_gpu(c), i32(t), i32(base), n_nodes=i32(nn))
    check_attention(r, K.attention(q64, c, t, base, n_nodes=nn, sm=0.125), BF)
    assert (r["out"][1] == 0).all() and torch.isneginf(r["lse"][1]).all() and torch.isneginf(r["lse"][2, 3:]).all()


@pytest.mark.parametrize("N,G,D", [(5, 2, 128), (5, 4, 64), (48, 4, 128), (40, 4, 64)])
def test_nan_where_it_is_not_seen_and_where_it_is(N, G, D):
    base, P = [50, 70], 16
    rng, c, t, q, q64 = problem(7, base, N, 2, G, D, P, HF)
    par = trees(rng, 2, N) if N > 8 else None
    for which in ("k", "v"):
        for pos in range(base[0] + N, t.shape[1] * P):      # past the end
            if t[0, pos // P] >= 0:
                c[which][t[0, pos // P], :, pos % P] = 0x7f
    node = 2
    p = base[1] + node
    c["v"][t[1, p // P], 0, p % P, 3:5] = 0xff              # one node's value: its descendants see it
    p = base[0] + 4
    c["k"][t[0, p // P], 1, p % P, 1] = 0x7f                # one node's key
    want = K.attention(q64, c, t, base, par, sm=D ** -0.5)
    assert np.isnan(want[0]).any() and not np.isnan(want[0]).all()
    r = sv.spec_attention_q8(q, to_gpu(c), i32(t), i32(base), parents=None if par is None else i32(par))
    check_attention(r, want, HF)


def test_infinite_and_nan_queries_stay_in_their_rows():
    base = [80]
    rng, c, t, q, q64 = problem(8, base, 4, 1, 2, 64, 16, BF)
    q[0, 1, 0, 3] = float("inf")
    q[0, 2, 1, 0] = float("nan")
    q[0, 3] = 0.0
    q64 = q.double().cpu().numpy()
    r = sv.spec_attention_q8(q, to_gpu(c), i32(t), i32(base))
    assert torch.isnan(r["out"][0, 1, 0]).all() and torch.isnan(r["out"][0, 2, 1]).all()
    keep = np.ones((1, 4, 2), dtype=bool)
    keep[0, 1, 0] = keep[0, 2, 1] = False
    out, lse, absv, smax = K.attention(np.where(np.isfinite(q64), q64, 0), c, t, base, sm=0.125)
    got = r["out"].double().cpu().numpy()
    assert (np.abs(got - out) <= 2.0 ** -8 * absv + 1e-6)[keep].all()


@pytest.mark.parametrize("N", [3, 36])
def test_bad_pages_and_parents(N):
    base, P, H, G, D = [40, 40, 40, -3], 16, 1, 4, 128
    rng, c, t, q, q64 = problem(9, [40] * 4, N, H, G, D, P, BF)
    par = trees(rng, 4, N)
    t[1, 1] = 10 ** 6
    par[2, 2] = 2
    r = sv.spec_attention_q8(q, to_gpu(c), i32(t), i32(base), parents=i32(par))
    assert r["status"].tolist() == [0, sv.STATUS_BAD_PAGE, sv.STATUS_BAD_PARENT, sv.STATUS_BAD_PAGE]
    ref = K.attention(q64[:3], c, t[:3], base[:3], par[:3], sm=D ** -0.5)
    check_attention({k: r[k][:3] for k in ("out", "lse")}, ref, BF)


@pytest.mark.parametrize("N,G", [(2, 4), (16, 4)])
def test_strided_queries_streams_graphs_and_own_buffers(N, G):
    base, H, D = [200, 90, 33], 2, 64
    rng, c, t, q, q64 = problem(10, base, N, H, G, D, 32, BF)
    Hq = H * G
    fused = torch.zeros((3, N, Hq + 2 * H, D), dtype=BF, device=DEV)
    fused[:, :, :Hq] = q
    cache, tab, bs = to_gpu(c), i32(t), i32(base)
    want = sv.spec_attention_q8(q, cache, tab, bs)
    ref = K.attention(q64, c, t, base, sm=0.125)
    check_attention(want, ref, BF)
    same = lambda r: torch.equal(r["out"], want["out"]) and torch.equal(r["lse"], want["lse"])  # noqa: E731
    assert same(sv.spec_attention_q8(fused[:, :, :Hq], cache, tab, bs))
    odd = torch.empty(q.numel() + 1, dtype=BF, device=DEV)[1:].view_as(q).copy_(q)      # not on 16 bytes
    assert same(sv.spec_attention_q8(odd, cache, tab, bs))
    assert same(sv.spec_attention_q8(q.transpose(1, 2).contiguous().transpose(1, 2), cache, tab, bs))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        r = sv.spec_attention_q8(q, cache, tab, bs)
    side.synchronize()
    assert same(r)
    out = {k: torch.empty_like(v) for k, v in want.items()}
    ws = torch.full((sv.load_library().spec_attention_q8_workspace_size(3, N, Hq, H, D),), 0xff, dtype=torch.uint8, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sv.spec_attention_q8(q, cache, tab, bs, workspace=ws, out=out)
    for _ in range(3):
        for v in out.values():
            v.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert same(out)


def test_many_requests():
    rng = np.random.default_rng(11)
    base = rng.integers(0, 150, 300).tolist()
    rng, c, t, q, q64 = problem(11, base, 2, 1, 2, 64, 16, BF)
    r = sv.spec_attention_q8(q, to_gpu(c), i32(t), i32(base))
    check_attention(r, K.attention(q64, c, t, base, sm=0.125), BF)


def _torch_attention(q, k, v, sm):
    """One request's float64 attention of [R, D] rows over [L, D] (all visible)."""
    x = q.double() @ k.double().T * sm
    return torch.softmax(x, -1) @ v.double(), torch.logsumexp(x, -1)


@pytest.mark.parametrize("N,G", [(1, 8), (8, 8)])
def test_offsets_past_32_bits(N, G):
    """Pages at the end of a pool of more than 4 GB, and a cache long enough for many CTAs to share an item."""
    P, D, pages, L = 128, 128, 270000, 40000
    g = torch.Generator(device=DEV).manual_seed(3)
    pool = [torch.empty((pages, 1, P, D), dtype=torch.float8_e4m3fn, device=DEV) for _ in "kv"]
    scale = [torch.full((pages, 1), 2.0 ** -7, device=DEV) for _ in "kv"]
    W = -(-(L + N) // P)
    ids = (pages - 1 - torch.randperm(W, generator=g, device=DEV)).to(torch.int32)
    for x in pool:
        x[ids.long()] = (torch.randn((W, 1, P, D), generator=g, device=DEV) * 100).clamp(-448, 448).to(x.dtype)
    q = (torch.randn((1, N, G, D), generator=g, device=DEV) * 2).to(BF)
    cache = sv.Q8Cache(*pool, *scale)
    r = sv.spec_attention_q8(q, cache, ids[None], i32([L]))
    k, v = ((x[ids.long()].float() * 2.0 ** -7).reshape(-1, D) for x in pool)
    for n in (0, N - 1):
        o, lse = _torch_attention(q[0, n], k[:L + n + 1], v[:L + n + 1], D ** -0.5)
        assert (r["out"][0, n].double() - o).abs().max() <= 2.0 ** -9 * o.abs().max() + 2.0 ** -10
        assert (r["lse"][0, n].double() - lse).abs().max() <= 2.0 ** -17 * 30
    s = torch.rand((1, 1, W * P), generator=g, device=DEV)
    w = sv.spec_attention_weights_q8(q, r["lse"], cache, ids[None], i32([L]), s)["scores"]
    x = torch.exp(q[0].double().view(N * G, D) @ k[:L].double().T * D ** -0.5 - r["lse"].double().view(-1, 1)).sum(0)
    assert ((w[0, 0, :L].double() - s[0, 0, :L].double() - x).abs() <= 2.0 ** -17 * 30 * x + 2.0 ** -23).all()


WEIGHTS = [  # base, N, H, G, D, P, dtype, path
    ([0], 1, 1, 1, 64, 16, BF, False),
    ([0, 16, 33], 4, 2, 4, 128, 16, BF, True),
    ([200, 65, 1], 6, 2, 5, 128, 32, HF, True),
    ([500], 6, 1, 8, 64, 64, BF, False),
    ([90, 64], 5, 2, 13, 128, 128, HF, True),                       # 65 rows: a second pass over the keys
    ([70], 12, 1, 16, 64, 16, BF, True),
]


@pytest.mark.parametrize("base,N,H,G,D,P,dtype,with_path", WEIGHTS)
def test_weights(base, N, H, G, D, P, dtype, with_path):
    rng, c, t, q, q64 = problem(20 + N, base, N, H, G, D, P, dtype)
    B, S = len(base), t.shape[1] * P + 5
    cache, tab, bs = to_gpu(c), i32(t), i32(base)
    lse = sv.spec_attention_q8(q, cache, tab, bs)["lse"]
    path = n_acc = None
    if with_path:
        n_acc = rng.integers(-1, N, B)
        n_acc[0] = N - 1
        path = np.stack([np.sort(rng.permutation(N)) for _ in range(B)])
    s = torch.from_numpy(rng.random((B, H, S)).astype(np.float32)).to(DEV)
    kw = dict(path_nodes=i32(path), num_accepted=i32(n_acc)) if with_path else {}
    r = sv.spec_attention_weights_q8(q, lse, cache, tab, bs, s, decay=0.5, **kw)
    want, err = K.weights(q64, lse.double().cpu().numpy(), c, t, base, s.double().cpu().numpy(), path, n_acc, D ** -0.5, 0.5)
    got = r["scores"].double().cpu().numpy()
    assert (np.abs(got - want) <= 2.0 ** -17 * err + 2.0 ** -22 * np.abs(want)).all()
    assert r["status"].tolist() == [0] * B
    in_place = s.clone()
    sv.spec_attention_weights_q8(q, lse, cache, tab, bs, in_place, decay=0.5, out={"scores": in_place, "status": r["status"]}, **kw)
    assert torch.equal(in_place, r["scores"])


def test_weights_sum_to_the_number_of_rows():
    base = [333, 50]
    rng, c, t, q, q64 = problem(31, base, 3, 2, 4, 128, 16, BF)
    cache, tab, bs = to_gpu(c), i32(t), i32(base)
    lse = sv.spec_attention_q8(q, cache, tab, bs)["lse"]
    s = torch.zeros((2, 2, t.shape[1] * 16), device=DEV)
    w = sv.spec_attention_weights_q8(q, lse, cache, tab, bs, s)["scores"]
    assert (w.sum(-1) - 3 * 4).abs().max() < 12 * 2.0 ** -17 * 30


def test_weights_of_bad_requests():
    base = [40, 40, 40]
    rng, c, t, q, q64 = problem(32, base, 3, 1, 4, 64, 16, BF)
    cache, bs = to_gpu(c), i32(base)
    lse = sv.spec_attention_q8(q, cache, i32(t), bs)["lse"]
    t[1, 0] = -1
    path = np.array([[0, 1, 2], [0, 1, 2], [0, 7, 2]])
    s = torch.rand((3, 1, 48), device=DEV)
    r = sv.spec_attention_weights_q8(q, lse, cache, i32(t), bs, s, path_nodes=i32(path), num_accepted=i32([2, 2, 2]))
    assert r["status"].tolist() == [0, sv.STATUS_BAD_PAGE, sv.STATUS_BAD_PAGE]
    assert torch.equal(r["scores"][1, 0, :16], s[1, 0, :16]) and torch.isfinite(r["scores"]).all()


@pytest.mark.parametrize("offset", [0.0, -60.0, 60.0])
@pytest.mark.parametrize("N,G,dtype,D", [(1, 2, BF, 64), (6, 4, BF, 128), (6, 2, HF, 64), (9, 4, BF, 64)])
def test_first_positions_on_no_page(N, G, dtype, D, offset):
    """A request whose first 128 positions have no page (a prefix that was dropped), and some later ones: the rest is
    attended to as if alone, however high or low its scores. Enough requests that a CTA has several tiles of one."""
    B, P = 240, 64
    base = [500] * B
    rng, c, t, q, q64 = problem(40 + N, base, N, 2, G, D, P, dtype, q_std=1.0)
    c["k"][..., 0], c["ks"][:] = K.encode(128.0), 2.0 ** -7      # every key begins with 1
    q[..., 0] = offset * D ** 0.5                               # so that this adds `offset` to every score
    q64 = q.double().cpu().numpy()
    t[:, :2] = -1
    t[::3, 2] = -1
    r = sv.spec_attention_q8(q, to_gpu(c), i32(t), i32(base))
    check_attention(r, K.attention(q64, c, t, base, sm=D ** -0.5), dtype)
    assert r["status"].tolist() == [sv.STATUS_BAD_PAGE] * B


@pytest.mark.parametrize("N,D,dtype,tree", [(992, 64, BF, False), (993, 64, HF, True), (1000, 128, BF, False), (1024, 128, HF, False),
                                            (1024, 128, BF, True), (1024, 64, BF, True)])
def test_most_nodes_of_a_single_head(N, D, dtype, tree):
    """One query head a kv head, so that a block's 128 rows are 128 nodes, up to the most nodes there can be."""
    base = [70]
    rng, c, t, q, q64 = problem(50, base, N, 1, 1, D, 64, dtype)
    par = np.array([[-1] + [int(rng.integers(0, n)) for n in range(1, N)]]) if tree else None
    r = sv.spec_attention_q8(q, to_gpu(c), i32(t), i32(base), parents=None if par is None else i32(par))
    check_attention(r, K.attention(q64, c, t, base, par, sm=D ** -0.5), dtype)
    assert r["status"].tolist() == [0]


def test_dimensions_of_one_have_any_stride():
    base = [40]
    rng, c, t, q, q64 = problem(51, base, 1, 1, 4, 64, 16, BF)
    cache, tab, bs = to_gpu(c), i32(t), i32(base)
    odd = q.as_strided(q.shape, (3, 5, 64, 1))
    r = sv.spec_attention_q8(odd, cache, tab, bs)
    check_attention(r, K.attention(q64, c, t, base, sm=0.125), BF)
    s = torch.zeros((1, 1, t.shape[1] * 16), device=DEV)
    w = [sv.spec_attention_weights_q8(x, r["lse"], cache, tab, bs, s)["scores"] for x in (q, odd)]
    assert torch.equal(*w)
    k = q[:, :, :1]
    caches = [to_gpu(c), to_gpu(c)]
    for x, into in zip((k.contiguous(), k.as_strided(k.shape, (3, 5, 7, 1))), caches):
        assert sv.spec_kv_append_q8(into, x, x, tab, bs)["status"].tolist() == [0]
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(*caches))


@pytest.mark.parametrize("N,G,D", [(4, 4, 64), (6, 2, 128), (20, 4, 64)])
def test_weights_of_rows_that_saw_nothing(N, G, D):
    """Rows past n_nodes, whose lse is -inf, give no weight where all rows are counted."""
    base = [40, 0, 70, 3]
    rng, c, t, q, q64 = problem(52, base, N, 2, G, D, 16, BF)
    cache, tab, bs, nn = to_gpu(c), i32(t), i32(base), i32([2, 0, N, 0])
    lse = sv.spec_attention_q8(q, cache, tab, bs, n_nodes=nn)["lse"]
    s = torch.from_numpy(rng.random((4, 2, t.shape[1] * 16)).astype(np.float32)).to(DEV)
    got = sv.spec_attention_weights_q8(q, lse, cache, tab, bs, s)
    want = sv.spec_attention_weights_q8(q, lse, cache, tab, bs, s, num_accepted=nn - 1)
    assert torch.isfinite(got["scores"]).all() and torch.equal(got["scores"], want["scores"])
    assert torch.equal(got["scores"][3, :, :3], s[3, :, :3])
    assert got["status"].tolist() == want["status"].tolist() == [0] * 4


def scale_problem(seed, B, N, H, G, D, P, dtype, tree=False):
    rng, c, t, q, q64 = problem(seed, [300 + 37 * b for b in range(B)], N, H, G, D, P, dtype)
    par = trees(rng, B, N) if tree else None
    return rng, c, t, q, q64, [300 + 37 * b for b in range(B)], par


@pytest.mark.parametrize("N,G,D,dtype", [(5, 3, 128, HF), (1, 2, 64, BF), (6, 4, 64, BF), (40, 2, 128, BF)])
def test_pages_of_zeros_and_pages_that_are_not_there(N, G, D, dtype):
    """A page of zeros has scale 2^-100. Pieces of a request that begin on a missing page, on such a page and on others
    count scales from different references, and weigh the same together all the same."""
    P, B = 16, 7
    rng, c, t, q, q64, base, _ = scale_problem(60, B, N, 3, G, D, P, dtype)
    q *= 0.05
    q64 = q.double().cpu().numpy()
    zero = rng.random(c["vs"].shape) < 0.3
    c["vs"][zero], c["v"][zero] = 2.0 ** -100, 0
    t[rng.random(t.shape) < 0.5] = -1
    r = sv.spec_attention_q8(q, to_gpu(c), i32(t), i32(base))
    check_attention(r, K.attention(q64, c, t, base, sm=D ** -0.5), dtype)


@pytest.mark.parametrize("missing", [0.0, 0.4])
@pytest.mark.parametrize("N,G,D,dtype", [(5, 3, 128, HF), (1, 2, 64, BF), (6, 4, 64, BF), (40, 2, 128, BF), (33, 3, 64, HF)])
def test_pages_of_scale_zero(N, G, D, dtype, missing):
    """Scales of zero beside pages of zeros as append writes them: their values are nothing, their weights count."""
    P, B = 16, 7
    rng, c, t, q, q64, base, par = scale_problem(61, B, N, 3, G, D, P, dtype, tree=N == 40)
    kind = rng.random(c["vs"].shape)
    c["vs"][kind < 0.6] = 2.0 ** -100
    c["v"][kind < 0.6] = 0
    c["vs"][kind < 0.3] = 0.0
    c["v"][kind < 0.15] = K.encode(100.0)
    t[rng.random(t.shape) < missing] = -1
    r = sv.spec_attention_q8(q, to_gpu(c), i32(t), i32(base), parents=None if par is None else i32(par))
    check_attention(r, K.attention(q64, c, t, base, par, sm=D ** -0.5), dtype)


@pytest.mark.parametrize("first", [True, False])
@pytest.mark.parametrize("N,G,D,dtype", [(5, 3, 128, BF), (1, 2, 64, BF), (40, 2, 128, BF), (33, 4, 64, BF)])
def test_pages_of_zeros_beside_large_values(N, G, D, dtype, first):
    """Values of 10^7 beside pages of zeros whose positions have scores some bits lower but are many."""
    P, B = 16, 5
    rng, c, t, q, q64, _, par = scale_problem(62, B, N, 2, G, D, P, dtype, tree=N == 40)
    base = [300 + 37 * b for b in range(B)]
    c["ks"][:], c["k"][..., :32] = 2.0 ** -7, K.encode(128.0)
    c["vs"][:] *= 2.0 ** 22
    q *= 0.05
    q[..., :32] = 9.0 / 32 * D ** 0.5              # a score of 9 where a key begins with ones, 0 where with zeros
    q64 = q.double().cpu().numpy()
    for b in range(B):                              # most pages hold zeros and score 13 bits lower
        for lp in range(base[b] // P):
            if (lp % 6 != 0) == first and lp > 0 or (lp == 0 and first):
                p = t[b, lp]
                c["v"][p], c["vs"][p], c["k"][p, :, :, :32] = 0, 2.0 ** -100, 0
    r = sv.spec_attention_q8(q, to_gpu(c), i32(t), i32(base), parents=None if par is None else i32(par))
    check_attention(r, K.attention(q64, c, t, base, par, sm=D ** -0.5), dtype)
