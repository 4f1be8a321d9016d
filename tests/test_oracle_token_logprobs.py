"""The log-prob oracle against scipy, and its gradient against differences."""

import numpy as np
from scipy.special import log_softmax

from oracle import token_logprobs as L


def test_values():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 50)) * 3
    x[1, 10:40] = -np.inf
    t = np.array([3, 2, -1, 49, 60])
    r = L.token_logprobs(x, t, T=0.7, n_top=4)
    lp = log_softmax(x / 0.7, axis=1)
    assert np.allclose(r["logprob"][[0, 1, 3]], lp[[0, 1, 3], [3, 2, 49]]) and r["logprob"][2] == 0
    p = np.exp(lp)
    assert np.allclose(r["entropy"], -(np.where(p > 0, p * np.where(p > 0, lp, 0), 0)).sum(1))
    assert r["status"].tolist() == [0, 0, 0, 0, 1]
    assert (r["top_tokens"][0] == np.argsort(-x[0])[:4]).all()


def test_rows_with_nothing_and_ties():
    x = np.full((2, 6), -np.inf)
    x[1, [1, 4]] = 2.0
    r = L.token_logprobs(x, np.array([0, 4]), n_top=3)
    assert r["lse"][0] == -np.inf and r["logprob"][0] == -np.inf and r["entropy"][0] == 0 and r["status"][0] == 4
    assert r["top_tokens"].tolist() == [[-1, -1, -1], [1, 4, -1]] and np.isclose(r["entropy"][1], np.log(2))


def test_gradient_by_differences():
    rng = np.random.default_rng(1)
    x, t, g, h = rng.standard_normal((3, 7)), np.array([2, -1, 6]), rng.standard_normal(3), rng.standard_normal(3)
    d = L.backward(x, t, g, h, T=1.3)
    for i in range(3):
        for j in range(7):
            e = np.zeros_like(x)
            e[i, j] = 1e-6
            f = [(lambda r: (g * r["logprob"] + h * r["entropy"]).sum())(L.token_logprobs(x + s * e, t, T=1.3)) for s in (1, -1)]
            assert abs((f[0] - f[1]) / 2e-6 - d[i, j]) < 1e-7
