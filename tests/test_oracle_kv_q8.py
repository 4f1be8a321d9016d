"""The cache oracle against hand-worked values and torch's e4m3 conversions."""

import numpy as np
import torch

from oracle import kv_q8 as K


def test_codes_agree_with_torch():
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(np.isnan(K.VALUES), np.isnan(want))
    fine = ~np.isnan(want)
    assert np.array_equal(K.VALUES[fine], want[fine])
    g = torch.Generator().manual_seed(1)
    x = torch.cat([torch.randn(5000, generator=g) * 10.0 ** torch.randint(-4, 3, (5000,), generator=g),
                   (torch.from_numpy(want[:126]) + torch.from_numpy(want[1:127])) / 2]).clamp(-448, 448)   # ties too
    assert np.array_equal(K.encode(x.numpy()), x.to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    assert K.encode([np.nan, np.inf, -np.inf, 0.0]).tolist() == [0x7f, 0x7e, 0xfe, 0]


def test_scale_is_the_smallest_power_of_two():
    assert K.need_scale([448.0]) == 1.0 and K.need_scale([448.01]) == 2.0 and K.need_scale([-224.0]) == 0.5
    assert K.need_scale([0.0]) == 2.0 ** -100 and K.need_scale([1e-45]) == 2.0 ** -100
    assert K.need_scale([np.inf, np.nan, 3.5]) == 2.0 ** -7


def _cache(pages, H, P, D):
    z = np.zeros((pages, H, P, D), dtype=np.uint8)
    return dict(k=z, v=z.copy(), ks=np.ones((pages, H)), vs=np.ones((pages, H)))


def test_append_grows_a_page_scale_and_keeps_its_values():
    c = _cache(2, 1, 16, 64)
    k = np.full((1, 3, 1, 64), 3.5)
    c, n, st = K.append(c, k, k, np.array([[1]]), [0])
    assert n.tolist() == [3] and st.tolist() == [0] and c["ks"][1, 0] == 2.0 ** -7
    c, n, _ = K.append(c, k * 256, k, np.array([[1]]), [3])
    assert c["ks"][1, 0] == 2.0 and c["vs"][1, 0] == 2.0 ** -7
    assert (K.decode(c["k"][1, 0, :3]) * 2 == 3.5).all() and (K.decode(c["k"][1, 0, 3:6]) * 2 == 896).all()


def test_attention_of_uniform_scores_is_a_mean_and_trees_hide_siblings():
    c = _cache(2, 1, 16, 64)
    rng = np.random.default_rng(0)
    v = rng.standard_normal((1, 5, 1, 64))
    c, _, _ = K.append(c, np.zeros((1, 5, 1, 64)), v, np.array([[0]]), [0])
    vals = K.decode(c["v"][0, 0, :5]) * c["vs"][0, 0]
    q = rng.standard_normal((1, 3, 2, 64))
    out, lse, _, _ = K.attention(q, c, np.array([[0]]), [2], parents=np.array([[-1, 0, 0]]))
    assert np.allclose(out[0, 1, 0], vals[:4].mean(0)) and np.allclose(lse[0, 1], np.log(4))
    assert np.allclose(out[0, 2, 1], vals[[0, 1, 2, 4]].mean(0))


def test_eviction_moves_the_kept_tail_into_holes():
    c = _cache(4, 1, 16, 64)
    for j in range(32):
        c["k"][j // 16, 0, j % 16] = j + 1
    c["ks"][:, 0] = [1.0, 2.0, 1.0, 1.0]
    scores = np.ones((1, 1, 64))
    scores[0, 0, [3, 5]] = 0.0
    scores[0, 0, 18:32] = 0.0
    pos = np.arange(64)[None, None]
    d, s, p, n, st = K.evict(c, np.array([[0, 1, -1, -1]]), [32], scores, pos, 16)
    assert n.tolist() == [16] and p[0, 0, 3] == 16 and p[0, 0, 5] == 17 and p[0, 0, 16] == -1
    assert d["ks"][0, 0] == 2.0 and d["k"][0, 0, 3, 0] == 17
    assert K.decode(d["k"][0, 0, 7, 0]) == K.VALUES[8] / 2   # a kept row under the grown scale
