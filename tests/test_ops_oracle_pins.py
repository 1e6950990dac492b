"""Closed forms that pin the fp64 oracles of the linear attention, the draft
verification and the block norms."""

import numpy as np

from oracle import ops_oracle as oo


def test_linear_without_decay_is_causal_attention_without_softmax():
    rng = np.random.default_rng(1)
    q, k, v = (rng.standard_normal((9, 2, 4)) for _ in range(3))
    got = oo.linear(q, k, v, np.zeros(2), 0.5, 2, 2)
    for h in range(2):
        want = 0.5 * np.tril(q[:, h] @ k[:, h].T) @ v[:, h]
        np.testing.assert_allclose(got["o"][:, h], want, atol=1e-13)
        np.testing.assert_allclose(got["final"][0, h], k[:, h].T @ v[:, h], atol=1e-13)


def test_linear_decay_two_tokens_by_hand():
    # S0 = 3, alpha = 1/2: S1 = 1.5 + 2*5 = 11.5, o1 = 11.5; S2 = 5.75 + 1*4 = 9.75, o2 = 2 * 9.75
    one = np.ones((2, 1, 1))
    got = oo.linear(one * [[[1]], [[2]]], one * [[[2]], [[1]]], one * [[[5]], [[4]]], np.log([0.5]), 1.0, 1, 1,
                    initial_state=np.full((1, 1, 1, 1), 3.0))
    np.testing.assert_allclose(got["o"].ravel(), [11.5, 19.5])
    np.testing.assert_allclose(got["final"].ravel(), [9.75])


def test_linear_forgets_at_minus_infinity():
    rng = np.random.default_rng(2)
    q, k, v = (rng.standard_normal((5, 1, 3)) for _ in range(3))
    g = np.zeros((5, 1))
    g[3] = -np.inf
    whole, tail = oo.linear(q, k, v, g, 1.0, 1, 1), oo.linear(q[3:], k[3:], v[3:], g[3:], 1.0, 1, 1)
    np.testing.assert_allclose(whole["o"][3:], tail["o"])


def test_verify_by_hand():
    p = np.array([[0.5, 0.5, 0.0], [0.25, 0.25, 0.5], [0.0, 0.5, 0.5]])
    q = np.array([[1.0, 0.0, 0.0], [0.0, 0.5, 0.5]])
    assert oo.verify_row(p, q, [0, 1], [0.49, 0.49, 0.5], 2) == ([0, 1, 2], 3)     # all accepted, c = 0, .5, 1
    assert oo.verify_row(p, q, [0, 1], [0.49, 0.5, 0.9], 2) == ([0, 0, -1], 2)     # .5 * .5 < .25 fails; rest at 0 only
    assert oo.verify_row(p, q, [0, 1], [0.5, 0.0, 0.0], 2) == ([1, -1, -1], 1)
    assert oo.verify_row(p, q, [0, 1], [0.0, 0.0, 0.0], 0) == ([0, -1, -1], 1)     # no drafts: p_0
    assert oo.verify_row(p, None, [0, 2], [0.4, 0.5, 0.5], 2) == ([0, 1, -1], 2)   # rest .25 .25 at 0, 1
    assert oo.verify_row(p, q, [0, 1], [0.0, 0.0, 0.0], -1) == ([-1, -1, -1], 0)


def test_verification_keeps_the_target_distribution():
    rng = np.random.default_rng(3)
    p, q = rng.dirichlet(np.ones(5), 2), rng.dirichlet(np.ones(5), 1)
    n = 20000
    count = np.zeros(5)
    for x, u in zip(rng.choice(5, n, p=q[0]), rng.random((n, 2))):
        count[oo.verify_row(p, q, [x], u, 1)[0][0]] += 1
    # five standard deviations of a count of n draws
    assert np.all(np.abs(count / n - p[0]) < 5 * np.sqrt(p[0] * (1 - p[0]) / n))


def test_block_norm_by_hand():
    h, n, _ = oo.block_norm(np.array([[3.0, 4.0]]), np.array([[0.0, 0.0]]), "sigmoid", np.array([[1.0, 1.0]]), 2.0,
                            np.array([1.0, 2.0]), np.array([1.0, 1.0]), 0.0)
    r = np.sqrt(12.5)
    np.testing.assert_allclose(h, [[1 + 3 / r, 1 + 8 / r]])
    np.testing.assert_allclose(n, h / np.sqrt((h ** 2).mean()))
    h, _, _ = oo.block_norm(np.array([[3.0, 4.0, 0.0, 2.0]]), post=np.ones(2), eps=0.0)
    np.testing.assert_allclose(h, [[3 / r, 4 / r, 0, np.sqrt(2)]])
