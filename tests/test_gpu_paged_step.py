"""A verify step on the 16-bit cache: append, attention, verification and the move of the accepted path, together."""

import os
import sys

import numpy as np
import pytest
import torch

import speculative_decoding_verification_72_gb300 as sv
from paged_utils import DEV, i32, inv_freq, normal, table

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def test_a_moved_path_is_as_if_it_alone_had_been_written():
    """Keys are rotated by depth, so rows moved by spec_kv_compact are bit for bit those of a chain written there."""
    rng = np.random.default_rng(0)
    B, N, H, D, P = 3, 8, 2, 128, 16
    base, f = [13, 0, 40], torch.from_numpy(inv_freq(D)).to(DEV)
    par = np.tile([-1, 0, 0, 1, 1, 2, 3, 3], (B, 1))
    path = np.array([[0, 2, 5, -1], [0, 1, 3, 7], [0, -1, -1, -1]])
    n_acc = [2, 3, 0]
    tab = i32(table(rng, [b + N for b in base], P, 12))
    k, v, q = (normal(rng, (B, N, h, D), torch.bfloat16)[1] for h in (H, H, 4 * H))
    one, two = sv.paged_cache(12, H, P, D), sv.paged_cache(12, H, P, D)
    r = sv.spec_kv_append_rope(one, k, v, tab, i32(base), f, q=q, parents=i32(par))
    for kv in one:
        n = sv.spec_kv_compact(kv, tab, i32(base), i32(path), i32(n_acc), N)
    take = i32(np.maximum(path, 0)).long()[:, :, None, None]
    pick = lambda t: t.gather(1, take.expand(-1, -1, t.shape[2], D))  # noqa: E731
    c = sv.spec_kv_append_rope(two, pick(k), pick(v), tab, i32(base), f, q=pick(q), n_nodes=i32([a + 1 for a in n_acc]))
    assert n["out_len"].tolist() == c["out_len"].tolist() == [16, 4, 41]
    for b in range(B):
        for s in range(base[b], int(n["out_len"][b])):
            at = (int(tab[b, s // P]), s % P)
            assert torch.equal(one.k[at], two.k[at]) and torch.equal(one.v[at], two.v[at])
        assert torch.equal(pick(r["q"])[b, :n_acc[b] + 1], c["q"][b, :n_acc[b] + 1])


def test_the_tree_pass_gives_what_the_chain_pass_gives():
    """The rows of one path of a tree see what the same rows see as a chain; sums run in another order."""
    rng = np.random.default_rng(1)
    B, N, H, G, D, P = 2, 12, 2, 4, 64, 16
    base, f = i32([100, 33]), torch.from_numpy(inv_freq(D)).to(DEV)
    par = np.tile([-1, 0, 0, 0, 2, 2, 4, 4, 6, 6, 8, 9], (B, 1))
    path = [0, 2, 4, 6, 8, 10]
    tab = i32(table(rng, [112, 45], P, 20))
    k, v, q = (normal(rng, (B, N, h, D), torch.bfloat16)[1] for h in (H, H, G * H))
    cache = sv.PagedCache(*(normal(rng, (20, P, H, D), torch.bfloat16)[1] for _ in "kv"))
    chain = sv.PagedCache(*(t.clone() for t in cache))
    r = sv.spec_kv_append_rope(cache, k, v, tab, base, f, q=q, parents=i32(par))
    a = sv.spec_attention(r["q"], cache, tab, base, parents=i32(par), softcap=10.0, window=60)
    c = sv.spec_kv_append_rope(chain, k[:, path], v[:, path], tab, base, f, q=q[:, path])
    b = sv.spec_attention(c["q"], chain, tab, base, softcap=10.0, window=60)
    # rounding of P (bf16, twice 2^-8) and of both outputs, of values of size 1 weighed down to less than 4 in all
    assert torch.equal(r["q"][:, path], c["q"])
    assert (a["out"][:, path].float() - b["out"].float()).abs().max() < 4 * 4 * 2.0 ** -8
    assert (a["lse"][:, path] - b["lse"]).abs().max() < 1e-4


def test_example():
    import paged_verify_step as E
    model = E.Model()
    prompt = torch.randint(0, model.vocab, (3, 190), generator=torch.Generator().manual_seed(5), dtype=torch.int32).cuda()
    plain, passes, _ = E.decode(model, prompt, 20)
    tokens, fewer, d = E.decode(model, prompt, 20, guesses=plain.int().cuda())
    assert tokens.shape == (3, 20) and fewer < passes
    assert (d.length.cpu() >= 189 + 20).all()
    # Sums run in another order where tokens come in other passes, so a near tie may fall the other way; few do.
    assert (tokens[:, :6] == plain[:, :6]).float().mean() > 0.8
