"""GPU parity of writing to and evicting from the 8-bit cache against oracle/kv_q8.py (exact)."""

import numpy as np
import pytest
import torch

import speculative_decoding_verification_72_gb300 as sv
from oracle import kv_q8 as K
from q8_utils import DEV, host_cache, i32, rows, same_cache, table, to_gpu, to_host

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    sv.load_library()


def run_append(c, k, v, t, base, **kw):
    cache = to_gpu(c)
    r = sv.spec_kv_append_q8(cache, k, v, i32(t), i32(base), **kw)
    return to_host(cache), r["out_len"].tolist(), r["status"].tolist()


@pytest.mark.parametrize("base,N,H,D,P,dtype", [
    ([0], 1, 1, 64, 16, BF), ([15, 16, 17, 0], 6, 2, 128, 16, BF), ([5, 64, 63], 1, 3, 64, 64, HF),
    ([0, 100], 300, 2, 128, 32, F32), ([7], 129, 1, 128, 128, HF), ([33, 31], 65, 2, 64, 128, F32), ([3], 200, 2, 64, 16, BF)])
def test_append(base, N, H, D, P, dtype):
    rng = np.random.default_rng(N)
    lens = [b + N for b in base]
    pages = sum(-(-n // P) for n in lens) + 2
    c, t = host_cache(rng, pages, H, P, D, pow2=False), table(rng, lens, P, pages)
    k, k64 = rows(rng, (len(base), N, H, D), dtype, 3.0)
    v, v64 = rows(rng, (len(base), N, H, D), dtype, 1e-3)
    want, n, st = K.append(c, k64, v64, t, base)
    got, gn, gst = run_append(c, k, v, t, base)
    same_cache(got, want)
    assert gn == n.tolist() and gst == st.tolist() == [0] * len(base)


def test_append_special_values():
    rng = np.random.default_rng(1)
    c, t = host_cache(rng, 4, 1, 16, 64), np.array([[0, 1], [2, 3]])
    x = torch.zeros((2, 20, 1, 64), device=DEV)
    x[0, 0, 0, 0], x[0, 1, 0, 1], x[0, 2, 0, 2], x[0, 3, 0, 3] = float("inf"), float("nan"), float("-inf"), 449.0
    x[0, 16:] = 1e-30
    x[1, 0, 0, 0], x[1, 1, 0, 5], x[1, 17] = 3e38, -0.0, 1e-42
    x64 = x.double().cpu().numpy()
    want, _, _ = K.append(c, x64, x64, t, [0, 0])
    got, _, _ = run_append(c, x, x, t, [0, 0])
    same_cache(got, want)


def test_append_accepted_path_over_the_nodes():
    """All nodes, then the accepted ones again: what is kept is what appending the accepted rows alone would give,
    under a scale that may be larger."""
    rng = np.random.default_rng(2)
    base, N, P = [30, 7, 16], 20, 16
    lens = [b + N for b in base]
    c, t = host_cache(rng, 12, 2, P, 128), table(rng, lens, P, 12)
    k, k64 = rows(rng, (3, N, 2, 128), BF, 2.0)
    path = np.array([[0, 2, 9, 15, -1], [0, 1, 2, 3, 4], [0, -1, -1, -1, -1]])
    n_acc = [3, 4, 0]
    w1, _, _ = K.append(c, k64, -k64, t, base)
    want, n, _ = K.append(w1, k64, -k64, t, base, path, n_acc)
    cache = to_gpu(c)
    sv.spec_kv_append_q8(cache, k, -k, i32(t), i32(base))
    r = sv.spec_kv_append_q8(cache, k, -k, i32(t), i32(base), path_nodes=i32(path), num_accepted=i32(n_acc))
    same_cache(to_host(cache), want)
    assert r["out_len"].tolist() == [34, 12, 17] == n.tolist()


def test_append_refuses_a_bad_request_whole():
    rng = np.random.default_rng(3)
    base, N, P = [0, 14, -1, 20, 0], 6, 16
    c, t = host_cache(rng, 12, 1, P, 64), table(rng, [32] * 5, P, 12)
    t[1, 1] = 99
    k, k64 = rows(rng, (5, N, 1, 64), HF)
    path = np.tile(np.arange(N), (5, 1))
    path[4, 3] = N
    n_acc = [5, 5, 5, 12, 5]
    want, n, st = K.append(c, k64, k64, t, base, path, n_acc)
    got, gn, gst = run_append(c, k, k, t, base, path_nodes=i32(path), num_accepted=i32(n_acc))
    same_cache(got, want)
    assert gn == n.tolist() and gst == st.tolist() == [0] + [sv.STATUS_BAD_PAGE] * 4


def test_append_strided_rows_and_nothing_to_write():
    rng = np.random.default_rng(4)
    qkv, q64 = rows(rng, (2, 5, 8, 64), BF)
    c, t = host_cache(rng, 6, 2, 16, 64), table(rng, [25, 12], 16, 6)
    want, _, _ = K.append(c, q64[:, :, 4:6], q64[:, :, 6:8], t, [20, 7])
    got, _, _ = run_append(c, qkv[:, :, 4:6], qkv[:, :, 6:8], t, [20, 7])
    same_cache(got, want)
    got, n, st = run_append(c, qkv[:, :, 4:6], qkv[:, :, 6:8], t, [20, 7], num_accepted=i32([-1, -1]))
    same_cache(got, c)
    assert n == [20, 7] and st == [0, 0]


EVICT = [  # lengths, keep, H, D, P, protect
    ([17], 16, 1, 64, 16, False), ([40, 16, 0, 33], 32, 2, 128, 16, True), ([300, 257, 256], 256, 2, 64, 64, True),
    ([5000], 4096, 1, 128, 128, False), ([9000, 4097], 1024, 1, 64, 32, True),
]


def evict_problem(seed, lens, keep, H, D, P):
    rng = np.random.default_rng(seed)
    pages = sum(-(-n // P) for n in lens) + 2
    c = host_cache(rng, pages, H, P, D, pow2=seed % 2 == 0)
    t = table(rng, lens, P, pages, width=max(-(-max(lens) // P), keep // P))
    S = t.shape[1] * P
    s = np.exp(2 * rng.standard_normal((len(lens), H, S))).astype(np.float32)
    pos = rng.permuted(np.tile(np.arange(S), (len(lens), H, 1)), axis=-1).astype(np.int32)
    return rng, c, t, s, pos


def run_evict(c, t, lens, s, pos, keep, sinks=0, protect=None):
    cache = to_gpu(c)
    S, Q = torch.from_numpy(s).to(DEV), torch.from_numpy(pos).to(DEV)
    r = sv.spec_kv_evict_q8(cache, i32(t), i32(lens), S, Q, keep, sinks, None if protect is None else i32(protect))
    want, ws, wp, n, st = K.evict(c, t, lens, s, pos, keep, sinks, protect)
    same_cache(to_host(cache), want)
    assert np.array_equal(r["scores"].cpu().numpy(), ws, equal_nan=True)
    assert np.array_equal(r["positions"].cpu().numpy(), wp)
    assert r["out_len"].tolist() == n.tolist() and r["status"].tolist() == st.tolist()
    # in place
    cache = to_gpu(c)
    sv.spec_kv_evict_q8(cache, i32(t), i32(lens), S, Q, keep, sinks, None if protect is None else i32(protect),
                        out=dict(scores=S, positions=Q, out_len=r["out_len"], status=r["status"]))
    same_cache(to_host(cache), want)
    assert np.array_equal(S.cpu().numpy(), ws, equal_nan=True) and np.array_equal(Q.cpu().numpy(), wp)
    return r


@pytest.mark.parametrize("lens,keep,H,D,P,protect", EVICT)
def test_evict(lens, keep, H, D, P, protect):
    rng, c, t, s, pos = evict_problem(len(lens) + keep // 16, lens, keep, H, D, P)
    run_evict(c, t, lens, s, pos, keep, sinks=3, protect=[max(n - 8, 0) for n in lens] if protect else None)


@pytest.mark.parametrize("kind", ["equal", "few_values", "nan_inf", "negative", "all_protected"])
def test_evict_ties_and_special_scores(kind):
    lens, keep = [900, 650], 512
    rng, c, t, s, pos = evict_problem(7, lens, keep, 2, 64, 16)
    sinks = 0
    if kind == "equal":
        s[:] = 1.0
    elif kind == "few_values":
        s[:] = rng.integers(0, 3, s.shape)
        s[0, 0, ::7] = -0.0
    elif kind == "nan_inf":
        s[rng.random(s.shape) < 0.3] = np.nan
        s[rng.random(s.shape) < 0.2] = -np.inf
        s[rng.random(s.shape) < 0.1] = np.inf
    elif kind == "negative":
        s[:] = -s
    else:
        sinks = 10 ** 6
    run_evict(c, t, lens, s, pos, keep, sinks=sinks)


def test_evict_longer_than_the_keys_held_in_shared_memory():
    rng, c, t, s, pos = evict_problem(8, [45000], 40960 + 2048, 1, 64, 128)
    run_evict(c, t, [45000], s, pos, 40960 + 2048, sinks=4)


def test_evict_refuses_bad_pages():
    lens, keep = [100, 100, 5000], 64
    rng, c, t, s, pos = evict_problem(9, [100, 100, 100], keep, 1, 64, 16)
    t[1, 2] = -1
    r = run_evict(c, t, lens, s, pos, keep)
    assert r["status"].tolist() == [0, sv.STATUS_BAD_PAGE, sv.STATUS_BAD_PAGE]


def test_attention_does_not_depend_on_the_order_of_slots():
    """Evicting, then attending, is attending to the kept tokens."""
    rng = np.random.default_rng(10)
    n, keep, P = 100, 64, 16
    c, t = host_cache(rng, 8, 1, P, 64), table(rng, [n], P, 8)
    c["ks"][:], c["vs"][:] = 2.0 ** -7, 2.0 ** -6          # one scale: no rescaling
    s = rng.random((1, 1, 112)).astype(np.float32)
    pos = np.arange(112, dtype=np.int32)[None, None]
    cache = to_gpu(c)
    r = sv.spec_kv_evict_q8(cache, i32(t), i32([n]), torch.from_numpy(s).to(DEV), torch.from_numpy(pos).to(DEV), keep)
    kept = np.sort(r["positions"].cpu().numpy()[0, 0, :keep])
    assert np.array_equal(kept, np.sort(np.argsort(-s[0, 0, :n], kind="stable")[:keep]))
    q, q64 = rows(rng, (1, 1, 2, 64), HF)
    # the query's own slot: keep - 1 is base, so every kept token is seen
    got = sv.spec_attention_q8(q, cache, i32(t), i32([keep - 1]))["out"].double().cpu().numpy()
    k = np.concatenate([K.decode(c["k"][p, 0]) for p in t[0]])[kept] * 2.0 ** -7
    v = np.concatenate([K.decode(c["v"][p, 0]) for p in t[0]])[kept] * 2.0 ** -6
    x = q64[0, 0] @ k.T * 0.125
    p = np.exp(x - x.max(1, keepdims=True))
    assert np.abs(got[0, 0] - p / p.sum(1, keepdims=True) @ v).max() < 2.0 ** -9 * 2


def test_evict_several_heads_past_the_keys_held_in_shared_memory():
    """Marks past the keys that fit lie in the list of rows itself, which each slot's thread overwrites: with several
    heads and requests the rows there are far past a head's slots, and a budget that ends inside the last batch of slots
    has threads with nothing to fetch beside others that write."""
    lens, keep = [45000, 43100], 43072          # 43072 = 10 * 4096 + 2112
    rng, c, t, s, pos = evict_problem(12, lens, keep, 3, 64, 64)
    c["ks"][:], c["vs"][:] = 2.0 ** -7, 2.0 ** -6
    run_evict(c, t, lens, s, pos, keep, sinks=4, protect=[n - 100 for n in lens])


@pytest.mark.parametrize("sinks,protect", [(10 ** 12, None), (-10 ** 12, None), (0, 2 ** 63 - 1), (0, -2 ** 63), (0, 2 ** 32 + 150)])
def test_evict_integers_past_32_bits(sinks, protect):
    lens, keep = [200], 64
    rng, c, t, s, pos = evict_problem(13, lens, keep, 1, 64, 16)
    want = K.evict(c, t, lens, s, pos, keep, sinks, None if protect is None else [protect])
    r = sv.spec_kv_evict_q8(to_gpu(c), i32(t), i32(lens), torch.from_numpy(s).to(DEV), torch.from_numpy(pos).to(DEV), keep, sinks,
                            None if protect is None else torch.tensor([protect], device=DEV))
    assert np.array_equal(r["positions"].cpu().numpy(), want[2])


def test_lengths_past_32_bits_are_out_of_range():
    rng = np.random.default_rng(14)
    c, t = host_cache(rng, 4, 1, 16, 64), table(rng, [20, 20], 16, 4)
    k, k64 = rows(rng, (2, 4, 1, 64), BF)
    cache = to_gpu(c)
    r = sv.spec_kv_append_q8(cache, k, k, i32(t), torch.tensor([2 ** 32 + 5, -2 ** 32 + 5]))
    assert r["status"].tolist() == [sv.STATUS_BAD_PAGE] * 2
    same_cache(to_host(cache), c)


@pytest.mark.parametrize("outlier", [1.0, 300.0, 1e4])
def test_what_a_rejected_node_leaves_behind(outlier):
    """All nodes and then the accepted ones, against the accepted ones alone: pages that begin with new rows are the same;
    the page that also holds earlier positions may have a larger scale, never a smaller one, and its values then differ by
    the two roundings (2^-4 of the value each, half of the smallest step under each scale)."""
    rng = np.random.default_rng(15)
    base, N, P, D = [20, 13], 24, 16, 64
    lens = [b + N for b in base]
    c, t = host_cache(rng, 10, 2, P, D), table(rng, lens, P, 10)
    k, _ = rows(rng, (2, N, 2, D), BF)
    k[:, 1] *= outlier                                         # node 1 lies in the page of base and is rejected
    path, n_acc = np.array([[0] + list(range(2, 22))] * 2), [20, 20]
    acc = torch.stack([k[b, path[b]] for b in range(2)])
    both, alone = to_gpu(c), to_gpu(c)
    sv.spec_kv_append_q8(both, k, -k, i32(t), i32(base))
    r = sv.spec_kv_append_q8(both, k, -k, i32(t), i32(base), path_nodes=i32(path), num_accepted=i32(n_acc))
    w = sv.spec_kv_append_q8(alone, acc, -acc, i32(t), i32(base))
    assert r["out_len"].tolist() == w["out_len"].tolist() == [b + 21 for b in base]
    a, b = to_host(both), to_host(alone)
    for codes, scales in (("k", "ks"), ("v", "vs")):
        for req, n in enumerate(b + 21 for b in base):
            for lp in range(-(-n // P)):
                page, m, first = t[req, lp], min(P, n - lp * P), lp == base[req] // P
                s, s0 = a[scales][page], b[scales][page]
                x = K.decode(a[codes][page, :, :m]) * s[:, None, None]
                y = K.decode(b[codes][page, :, :m]) * s0[:, None, None]
                if not first:
                    assert np.array_equal(s, s0) and np.array_equal(a[codes][page, :, :m], b[codes][page, :, :m])
                    continue
                assert (s >= s0).all() and ((s > s0).all() if outlier > 100 else True)
                big = np.maximum(np.abs(x), np.abs(y))
                assert (np.abs(x - y) <= 2.0 ** -3 * big + 2.0 ** -10 * (s + s0)[:, None, None]).all()
