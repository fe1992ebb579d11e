"""The tolerance of the drafted trees' values is narrow enough: in float64, a
large value row that is lost, doubled or replaced by its neighbour moves some
output of every row that sees it by more than twice what it may be off (no
GPU)."""
import numpy as np
import pytest

from _tree_util import borders, reference
from oracle.tree import tree_attention, tree_mask

EPS = {"bf16": 2.0 ** -7, "f16": 2.0 ** -10}


@pytest.mark.parametrize("eps", list(EPS))
@pytest.mark.parametrize("n,ctx,window", [
    (7, 30, -1), (20, 600, -1), (12, 900, 200), (5, 3, 2)])
def test_a_misplaced_row_shows(n, ctx, window, eps):
    rng = np.random.default_rng(n)
    eps, d = EPS[eps], 64
    L = ctx + n
    par = [-1] + [int(rng.integers(max(0, i - 4), i)) for i in range(1, n)]
    # (short queries: no key's weight is far below the others')
    q, k = rng.standard_normal((n, 2, d)) / 4, rng.standard_normal((L, 1, d))
    v = rng.standard_normal((L, 1, d))
    marks = borders(par, ctx, L, window)
    v[marks] *= 64
    out, _, tol, _ = reference(q, k, v, par, eps, d ** -0.5, window=window)
    seen = tree_mask(par, ctx, L, window)
    assert seen[:, marks].any()

    def shows(w, rows):
        moved, _ = tree_attention(q, k, w, par, d ** -0.5, window_left=window)
        # (of some head)
        return (np.abs(moved - out) > 2 * tol).any(-1)[rows].all()
    for j in marks:
        rows = np.flatnonzero(seen[:, j])
        if not len(rows):
            continue
        for factor in (0.0, 2.0):
            w = v.copy()
            w[j] *= factor
            assert shows(w, rows), (j, factor)
        w = v.copy()
        w[j] = v[j - 1 if j else 1]
        assert shows(w, rows), j
