"""Pins of the float64 reference of a speculative decoding step (no GPU):
cases worked out by hand, and its agreement with the causal reference."""
import numpy as np
import pytest

from _util import random_case
from oracle import paged_attention_ref
from oracle.tree import (ancestors, compact, tree_attention, tree_mask,
                         verify)

#      0
#     / \
#    1   2        3 under 1, 4 and 5 under 2
TREE = [-1, 0, 0, 1, 2, 2]


def test_ancestors():
    assert ancestors(TREE, 5) == [5, 2, 0]
    assert ancestors(TREE, 3) == [3, 1, 0]
    assert ancestors(TREE, 0) == [0]


def test_mask_of_a_tree():
    got = tree_mask(TREE, 2, 8)
    want = np.zeros((6, 8), bool)
    want[:, :2] = True
    for i, way in enumerate(([0], [0, 1], [0, 2], [0, 1, 3], [0, 2, 4],
                             [0, 2, 5])):
        want[i, [2 + w for w in way]] = True
    assert (got == want).all()


def test_mask_of_a_window():
    # row 5 at position 4: keys 3 and 4 in a window of one; of its ancestors
    # (position 3: row 2, position 2: row 0) the parent
    got = tree_mask(TREE, 2, 8, window_left=1)
    assert np.flatnonzero(got[5]).tolist() == [4, 7]
    assert np.flatnonzero(got[0]).tolist() == [1, 2]
    assert np.flatnonzero(got[2]).tolist() == [2, 4]


def test_mask_without_context():
    # fewer keys than rows: the first rows' keys are missing
    got = tree_mask([-1, 0, 1], -1, 2)
    assert got.tolist() == [[False, False], [True, False], [True, True]]


@pytest.mark.parametrize("window,softcap,sink", [
    (-1, 0.0, False), (4, 0.0, False), (0, 0.0, True), (-1, 5.0, True)])
def test_a_chain_is_causal_attention(window, softcap, sink):
    rng = np.random.default_rng(0)
    q, ks, vs, kc, vc, table, cu, su = random_case(rng, [5, 1, 3], [9, 4, 3],
                                                   4, 2, 8)
    sinks = rng.standard_normal(4) if sink else None
    out, lse = paged_attention_ref(
        q, kc, vc, cu, su, table, 8 ** -0.5, causal=True,
        window_size=(window, -1), softcap=softcap, sinks=sinks)
    for b in range(3):
        n = cu[b + 1] - cu[b]
        o, l = tree_attention(q[cu[b]:cu[b + 1]], ks[b], vs[b],
                              np.arange(n) - 1, 8 ** -0.5, softcap, window,
                              sinks)
        np.testing.assert_allclose(o, out[cu[b]:cu[b + 1]], atol=1e-13)
        np.testing.assert_allclose(l, lse[:, cu[b]:cu[b + 1]], atol=1e-13)


def test_a_path_of_a_tree_is_its_own_chain():
    rng = np.random.default_rng(1)
    q = rng.standard_normal((6, 2, 8))
    k = rng.standard_normal((9, 1, 8))
    v = rng.standard_normal((9, 1, 8))
    out, lse = tree_attention(q, k, v, TREE, 0.3)
    way = [0, 2, 5]
    keys = [0, 1, 2] + [3 + w for w in way]
    o, l = tree_attention(q[way], k[keys], v[keys], [-1, 0, 1], 0.3)
    np.testing.assert_allclose(out[way], o, atol=1e-14)
    np.testing.assert_allclose(lse[:, way], l, atol=1e-14)


P = np.array([[.5, .25, .25, 0], [.1, .2, .3, .4], [0, 0, 1, 0]])


def test_verify_a_chain():
    # .2 < .5 stands, .2 < .4 stands, then row 2's only token
    assert verify(P, [9, 0, 3], [.9, .2, .2], [-1, 0, 1]) == ([0, 3, 2],
                                                              [0, 1, 2])
    # refused at once: token 0's mass is gone, .25 / .25 of .5 are left
    assert verify(P, [9, 0, 3], [.4, .7, .2], [-1, 0, 1]) == ([1], [0])
    assert verify(P, [9, 0, 3], [.6, .7, .2], [-1, 0, 1]) == ([2], [0])


def test_verify_siblings_renormalize():
    # token 0 refused (.6 >= .5); token 1 against .25 / .5
    tree = [-1, 0, 0]
    assert verify(P, [9, 0, 1], [0., .6, .49], tree) == ([1, 2], [0, 2])
    assert verify(P, [9, 0, 1], [0., .6, .51], tree) == ([2], [0])


def test_verify_with_draft_probabilities():
    q = np.array([[.75, .25, 0, 0]] * 3)
    # u q < p: .6 * .75 < .5 stands; .7 * .75 does not
    assert verify(P, [9, 0, 0], [.99, .6, .9], [-1, 0, 1], q)[1] == [0, 1]
    # then R = max(p - q, 0) = (0, 0, .25, 0)
    assert verify(P, [9, 0, 0], [.99, .7, .9], [-1, 0, 1], q) == ([2], [0])


@pytest.mark.parametrize("bad", [-.2, float("-inf"), float("nan")])
def test_verify_counts_a_negative_draft_probability_as_none(bad):
    p = np.array([[.5, .25, .25, 0], [1, 0, 0, 0], [1, 0, 0, 0]])
    q = np.array([[.75, bad, 0, bad]] * 3)
    # token 3, which neither has, does not stand
    assert verify(p[:2], [9, 3], [.6, .5], [-1, 0], q[:2]) == ([2], [0])
    # token 1, which the draft does not have, does
    assert verify(p[:2], [9, 1], [.6, .99], [-1, 0], q[:2]) == ([1, 0],
                                                               [0, 1])
    # what is left after token 0 is refused: (0, .25, .25, 0)
    tree = [-1, 0, 0]
    assert verify(p, [9, 0, 3], [.4, .9, 0.], tree, q) == ([1], [0])
    assert verify(p, [9, 0, 0], [.6, .9, .9], tree, q) == ([2], [0])


def test_verify_with_nothing_left():
    # the draft covers the target: R becomes nothing, the target stays
    q = np.ones((3, 4))
    assert verify(P, [9, 3, 0], [.6, .5, .9], [-1, 0, 1], q) == ([1], [0])
    none = np.zeros((1, 3))
    assert verify(none, [0], [.5], [-1]) == ([-1], [0])
    # a number of 1: the last token that can be
    assert verify(P[:1], [0], [1.0], [-1]) == ([2], [0])


def test_verify_keeps_the_target_distribution():
    """What the first position says is distributed as the target, whatever
    was drafted: exact for one drafted token, by integrating over its number
    and the last one's on a grid that meets every threshold."""
    p, q = np.array([.5, .3, .2]), np.array([.2, .3, .5])
    grid = (np.arange(1000) + .5) / 1000
    got = np.zeros(3)
    for x in range(3):
        stands = min(1.0, p[x] / q[x])
        got[x] += q[x] * stands
        if stands < 1:
            for u in grid:
                said, _ = verify([p, p], [0, x], [u, stands + 1e-9],
                                 [-1, 0], [q, q])
                got[said[0]] += q[x] * (1 - stands) / 1000
    np.testing.assert_allclose(got, p, atol=1e-3)


def test_compact():
    cache = np.arange(6 * 2).reshape(6, 2, 1, 1)
    out = compact(cache, np.array([4, 0, 2]), 1, [0, 2, 3])
    flat = [out[4, 0], out[4, 1], out[0, 0], out[0, 1], out[2, 0], out[2, 1]]
    assert [int(x[0, 0]) for x in flat] == [8, 9, 1, 4, 4, 5]
