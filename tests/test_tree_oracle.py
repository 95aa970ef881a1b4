"""The oracle of trees of drafted tokens against closed forms and against the oracle of causal windows."""

import numpy as np
import pytest

import oracle

tree = oracle.tree


def test_a_chain_is_a_causal_window():
    r = np.random.default_rng(0)
    B, Hq, Hkv, n, T, D = 3, 4, 2, 5, 40, 8
    q, k, v = r.standard_normal((B, Hq, n, D)), r.standard_normal((B, Hkv, T, D)), r.standard_normal((B, Hkv, T, D))
    parents = np.tile(np.arange(n) - 1, (B, 1))
    lens = [40, 17, 3]
    out, lse = tree.attend(q, k, v, parents, lens, None, 0.3)
    ro, rl = oracle.decode_rows(q, k, v, 0.3, causal=True, seq_lens=lens, max_seq_len=T)
    assert np.allclose(out, ro, rtol=0, atol=1e-13) and np.allclose(lse, rl, rtol=0, atol=1e-13)


def test_siblings_do_not_see_each_other():
    k = np.zeros((1, 1, 4, 2))
    v = np.arange(8.0).reshape(1, 1, 4, 2)
    out, lse = tree.attend(np.ones((1, 1, 3, 2)), k, v, np.array([[-1, 0, 0]]), [4], None, 1.0)
    assert np.array_equal(out[0, 0], [v[0, 0, :2].mean(0), v[0, 0, :3].mean(0), v[0, 0, [0, 1, 3]].mean(0)])
    assert np.allclose(lse[0, 0], np.log([2, 3, 3]))
    out, _ = tree.attend(np.ones((1, 1, 4, 2)), k, v, np.array([[9, -1, 0, 1]]), [4], [3], 1.0)  # one row of padding
    assert np.isnan(out[0, 0, 0]).all() and np.array_equal(out[0, 0, 3], v[0, 0].mean(0))


@pytest.mark.parametrize("drafted", [True, False])
def test_the_walk_gives_the_target_distribution(drafted):
    """Over a fine grid of random numbers the first new token has the target's probabilities, whatever the draft is."""
    p = np.array([[0.5, 0.25, 0.125, 0.125]] * 3)
    q = np.array([[0.125, 0.5, 0.25, 0.125]] * 3)
    parents = np.array([-1, 0, 0])
    steps = (np.arange(16) + 0.5) / 16
    got = np.zeros(4)
    pairs = [(a, b) for a in range(4) for b in range(4)] if drafted else [(1, 0)]
    for a, b in pairs:
        weight = q[0, a] * q[0, b] if drafted else 1.0
        for u1 in steps:
            for u2 in steps:
                for u0 in steps:
                    path, token = tree.verify([0, a, b], parents, p, [u0, u1, u2], q if drafted else None)
                    first = token if len(path) == 1 else [0, a, b][path[1]]
                    got[first] += weight / 16 ** 3
    assert np.abs(got - p[0]).max() < 0.05, got  # a grid of 16 in each number


def test_verify_by_hand():
    p = np.array([[0.6, 0.4], [0.1, 0.9], [1.0, 0.0]])
    assert tree.verify([0, 0, 1], [-1, 0, 1], p, [0.0, 0.59, 0.89]) == ([0, 1, 2], 0)
    assert tree.verify([0, 0, 1], [-1, 0, 1], p, [0.5, 0.61, 0.0]) == ([0], 1)
    assert tree.verify([0, 0, 0], [-1, 0, 0], p, [0.5, 0.61, 0.0]) == ([0], 1)  # the same word again is refused
    assert tree.verify([], [], p[:0], []) == ([], -1)
    # p = q: accepted below 1; a refusal leaves nothing, and the target itself is drawn from
    assert tree.verify([0, 0], [-1, 0], p, [0.7, 0.99], p) == ([0, 1], 1)
    assert tree.verify([0, 0], [-1, 0], p, [0.7, 1.0], p) == ([0], 1)


def test_keep():
    x = np.arange(2 * 1 * 6 * 1).reshape(2, 1, 6, 1)
    y = tree.keep(x, np.array([[0, 2, 3], [1, 9, 9]]), [1, 4], [3, 1])
    assert y[0, 0, :, 0].tolist() == [0, 1, 3, 4, 4, 5] and y[1, 0, :, 0].tolist() == [6, 7, 8, 9, 11, 11]
