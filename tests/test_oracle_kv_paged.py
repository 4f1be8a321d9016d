"""The 16-bit cache's oracle against closed forms and properties of the definitions."""

import numpy as np
import pytest

from oracle import kv_paged as K

rng = np.random.default_rng(0)


@pytest.mark.parametrize("interleaved", [False, True])
def test_turning_keeps_lengths_and_depends_on_distance_alone(interleaved):
    f = np.array([1.0, 0.3, 0.01, 1e-4], np.float32)
    x, y = rng.standard_normal((2, 1, 8)), rng.standard_normal((2, 1, 8))
    a = K.turn(x, [5, 105], f, interleaved)
    b = K.turn(y, [2, 102], f, interleaved)
    assert np.allclose(np.linalg.norm(a, axis=-1), np.linalg.norm(x, axis=-1))
    assert np.allclose((K.turn(x[:1], [7], f, interleaved) * K.turn(y[:1], [3], f, interleaved)).sum(),
                       (K.turn(x[:1], [1007], f, interleaved) * K.turn(y[:1], [1003], f, interleaved)).sum())
    assert a.shape == b.shape == x.shape


def test_turning_by_hand():
    f = np.array([np.pi / 2], np.float32)
    x = np.array([[[1.0, 0.0, 5.0]]])
    assert np.allclose(K.turn(x, [1], f), [[[0.0, 1.0, 5.0]]], atol=1e-7)
    assert np.allclose(K.turn(x, [2], f, True), [[[-1.0, 0.0, 5.0]]], atol=1e-6)


def test_a_row_that_sees_one_slot_gets_its_value():
    c = dict(k=rng.standard_normal((2, 4, 1, 3)), v=rng.standard_normal((2, 4, 1, 3)))
    q = rng.standard_normal((1, 1, 2, 3))
    out, lse, *_ = K.attention(q, c, np.array([[1]]), [0], sm=0.5)
    assert np.allclose(out[0, 0, 0], c["v"][1, 0, 0]) and np.isclose(lse[0, 0, 1], 0.5 * q[0, 0, 1] @ c["k"][1, 0, 0])
    out, lse, *_ = K.attention(q, c, np.array([[0, 1]]), [5], window=1)   # itself alone
    assert np.allclose(out[0, 0, 0], c["v"][1, 1, 0])


def test_a_chain_is_a_tree_of_one_path_and_zero_slopes_are_none():
    c = dict(k=rng.standard_normal((3, 4, 2, 4)), v=rng.standard_normal((3, 4, 2, 4)))
    t, q = np.array([[2, 0, 1]]), rng.standard_normal((1, 4, 4, 4))
    a = K.attention(q, c, t, [6], window=3, cap=2.0)
    b = K.attention(q, c, t, [6], parents=np.array([[-1, 0, 1, 2]]), window=3, cap=2.0, slopes=np.zeros(4))
    assert all(np.allclose(x, y) for x, y in zip(a, b))


def test_siblings_do_not_see_each_other_and_stand_at_one_position():
    c = dict(k=rng.standard_normal((2, 4, 1, 4)), v=rng.standard_normal((2, 4, 1, 4)))
    q = np.repeat(rng.standard_normal((1, 1, 1, 4)), 3, 1)
    par = np.array([[-1, 0, 0]])
    c["k"][0, 2], c["v"][0, 2] = c["k"][0, 1], c["v"][0, 1]
    out, lse, *_ = K.attention(q, c, np.array([[0]]), [0], parents=par, slopes=np.ones(1))
    assert np.allclose(out[0, 1], out[0, 2]) and np.allclose(lse[0, 1], lse[0, 2])
    cache, n, st, _ = K.append_rope(dict(k=np.zeros((1, 4, 1, 4)), v=np.zeros((1, 4, 1, 4))), np.ones((1, 3, 1, 4)),
                                    np.ones((1, 3, 1, 4)), np.array([[0]]), [0], np.array([1.0, 0.5]), parents=par)
    assert np.allclose(cache["k"][0, 1], cache["k"][0, 2]) and n[0] == 3 and st[0] == 0


def test_what_is_bad_is_left_alone():
    cache = dict(k=rng.standard_normal((2, 4, 1, 4)), v=rng.standard_normal((2, 4, 1, 4)))
    new = rng.standard_normal((3, 3, 1, 4))
    got, n, st, _ = K.append_rope(cache, new, new, np.array([[0, -1], [0, 7], [1, 0]]), [2, 6, 0], np.ones(1, np.float32),
                                  n_nodes=[3, 3, 0])
    assert np.array_equal(got["k"], cache["k"]) and n.tolist() == [2, 6, 0] and st.tolist() == [256, 256, 0]
    out, lse, *_ = K.attention(np.ones((1, 2, 1, 4)), cache, np.array([[-1]]), [0])
    assert (out == 0).all() and (lse == -np.inf).all()


def test_a_cap_bounds_scores():
    c = dict(k=100 * rng.standard_normal((1, 4, 1, 4)), v=rng.standard_normal((1, 4, 1, 4)))
    out, lse, *_ = K.attention(100 * np.ones((1, 1, 1, 4)), c, np.array([[0]]), [3], cap=1.0)
    assert np.abs(lse - np.log(4)).max() <= 1.0
