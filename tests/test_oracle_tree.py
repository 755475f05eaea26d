"""Pins of the oracle of a speculative step: brute force, closed forms and the laws it has to keep."""
import numpy as np
import pytest

import oracle
import split_kv_flash_decode_gb300 as fd


def test_ancestors_and_masks():
    parents = [-1, 0, 0, 1, 3, 2]
    sees = oracle.ancestors(parents)
    assert [list(np.flatnonzero(r)) for r in sees] == [[0], [0, 1], [0, 2], [0, 1, 3], [0, 1, 3, 4], [0, 2, 5]]
    masks, depths = fd.tree_masks(parents)
    assert masks == [1, 3, 5, 11, 27, 37] and depths == [0, 1, 1, 2, 3, 2]
    chain, deep = fd.tree_masks(range(-1, 63))
    assert chain[62] == 2 ** 63 - 1 and chain[63] == -1 and deep[63] == 63
    for bad in ([0], [-1, 1], [-1, -1], [-1, 0, 5], range(-1, 64)):
        with pytest.raises(ValueError):
            fd.tree_masks(bad)


def test_a_path_is_a_decode_of_its_tokens():
    """Every node's output is the decode of the prefix and its path alone."""
    rs = np.random.default_rng(0)
    lens, trees = [9, 4, 3], [[-1, 0, 0, 2], [-1, 0, 1, 2], []]
    sees = [oracle.ancestors(t) for t in trees]
    q = rs.standard_normal((8, 4, 8))
    k, v = rs.standard_normal((2, 16, 2, 8))
    out, lse = oracle.tree_reference(q, k, v, lens, sees)
    at = t = 0
    for L, s in zip(lens, sees):
        for i in range(len(s)):
            rows = [at + j for j in range(L - len(s))] + [at + L - len(s) + j for j in np.flatnonzero(s[i])]
            one, one_lse = oracle.decode_reference(q[t:t + 1], k[rows], v[rows], [len(rows)], "f64")
            assert np.allclose(out[t], one[0], rtol=1e-13, atol=1e-14) and np.allclose(lse[t], one_lse[0], rtol=1e-13)
            t += 1
        at += L


def test_a_token_that_sees_nothing():
    out, lse = oracle.tree_reference(np.ones((2, 1, 4)), np.ones((2, 1, 4)), np.ones((2, 1, 4)), [2],
                                     [np.array([[False, False], [False, True]])])
    assert (out[0] == 0).all() and lse[0, 0] == -np.inf and np.allclose(out[1], 1) and np.allclose(lse[1], 2.0)


def test_verdicts_by_hand():
    p = np.array([[0.5, 0.25, 0.25, 0], [0, 0, 1, 0], [0.125, 0.125, 0.25, 0.5]])
    # The root's children 0 (p 0.5) and 1 (0.25 of the 0.5 left).
    walk = lambda u: oracle.verify_walk(p, [9, 0, 1], u, [-1, 0, 0])  # noqa: E731
    assert walk([0.3, 0.499, 0]) == ([0, 1], [0, 2])
    assert walk([0.9, 0.5, 0.499]) == ([0, 2], [1, 3])
    assert walk([0.0, 0.5, 0.5]) == ([0], [2])
    # A chain that was drawn from q: u q < p; what is left of p over q.
    q = np.array([[9.0] * 4, [0.25, 0.5, 0.25, 0], [0.25, 0.25, 0.25, 0.25]])
    chain = lambda u, t: oracle.verify_walk(p, [3, *t], u, draft=q)  # noqa: E731
    assert chain([0.5, 0.49, 0.99], [1, 2]) == ([0, 1, 2], [1, 2, 3])   # 0.49 x 0.5 < 0.25, then 1 > 0.25
    assert chain([0.99, 0.5, 0.0], [1, 2]) == ([0], [0])                # left: 0.25 of token 0 alone
    assert chain([0.2, 0.49, 0.0], [1, 3]) == ([0, 1], [1, 2])          # p of token 3 is 0: never stands
    # Nothing left: from the target itself; nothing there either: -1.
    assert oracle.verify_walk(np.array([[1.0, 0]]), [0], [0.7]) == ([0], [0])
    assert oracle.verify_walk(np.array([[0.75, 0], [1, 0]]), [0, 0], [0.5, 0.8], [-1, 0]) == ([0], [0])
    assert oracle.verify_walk(np.array([[np.nan, -1.0]]), [0], [0.7]) == ([0], [-1])


@pytest.mark.parametrize("drawn", [False, True])
def test_the_first_token_follows_the_target(drawn):
    """Over all uniforms (a fine grid), the first token comes out with the target's probabilities."""
    p = np.array([0.4, 0.1, 0.3, 0.2])
    q = np.array([0.1, 0.5, 0.3, 0.1])
    got, grid = np.zeros(4), (np.arange(60) + 0.5) / 60
    for x, share in enumerate(q if drawn else [1.0]):
        target, tokens = np.tile(p, (3, 1)), [0, x, 2]
        for u in grid:
            for v in grid:
                for w in ([0.5] if drawn else grid[::4]):
                    _, said = oracle.verify_walk(target, tokens, [w if not drawn else v, u, v], *(
                        (None, np.tile(q, (3, 1))) if drawn else ([-1, 0, 0], None)))
                    got[said[0]] += share / (60 * 60 * (1 if drawn else 15))
    assert np.abs(got - p).max() < 0.02


def test_keep_rows():
    x = np.arange(6)
    assert list(oracle.keep_rows(x, [0, 2, 5])) == [0, 2, 5, 3, 4, 5]
    assert list(oracle.keep_rows(x, [1, 1])) == [1, 1, 2, 3, 4, 5]
    assert list(oracle.keep_rows(x, [2, 1, 3])) == [2, 1, 2, 3, 4, 5]
    assert list(oracle.keep_rows(x, [0, 6, 7])) == [0, 1, 2, 3, 4, 5]
    assert list(oracle.keep_rows(x, [-1])) == [0, 1, 2, 3, 4, 5]


def test_planted_mistakes_are_seen():
    """A wrong mask, a tried token that stays, a draw that takes the sum up to it as enough."""
    p = np.array([[0.5, 0.5], [0.5, 0.5], [0.5, 0.5]])
    right = oracle.verify_walk(p, [0, 0, 1], [0.0, 0.6, 0.99], [-1, 0, 0])
    assert right == ([0, 2], [1, 0])                       # 0.5 of 0.5: certain
    assert oracle.verify_walk(p, [0, 0, 1], [0.0, 0.6, 0.99], [-1, 0, 1]) != right
    rs = np.random.default_rng(1)
    q, k = rs.standard_normal((3, 1, 4)), rs.standard_normal((5, 1, 4))
    a = oracle.tree_reference(q, k, k, [5], [oracle.ancestors([-1, 0, 0])])[0]
    b = oracle.tree_reference(q, k, k, [5], [oracle.ancestors([-1, 0, 1])])[0]
    assert np.allclose(a[:2], b[:2]) and not np.allclose(a[2], b[2], atol=1e-3)
