"""How far an attention output over drafted trees may be off, from its
arithmetic, and which value rows to make large so that a misplaced one shows."""
import numpy as np

from oracle.tree import tree_attention, tree_mask


def reference(q, k, v, parents, eps, scale, softcap=0.0, window=-1,
              sinks=None):
    """One request in float64: out, lse, and what either may be off.

    With A = sum p |v| (p: the probabilities), an output moves by
    * expm1(2 d) A: the logits are off by d, at most (D + 8) float32 roundings
      of the largest sum of their terms' magnitudes and 32 of the cap;
    * eps / 2 A: the probabilities round to the call's type.  f16 holds them
      at 2^11 of the row's reference maximum, whose own is in their sum, and
      steps of 2^-24: 2^-36 of it a key and |v|;
    * 2^-23 A a key: products of 16 keys add up to a float32 sum (17 roundings
      of it and their alignment: 2^-20), sums of the probabilities in eighths,
      rescaled every 64 keys at most;
    * 2^-18 A: exponentials (2^-22 each) and the joins of streams and pieces;
    * its own rounding, eps / 2, or 2^-25 below f16's normal numbers."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    out, lse = tree_attention(q, k, v, parents, scale, softcap, window, sinks)
    alive = np.where(np.isneginf(lse), 0.0, lse)
    if not len(k):          # (zeros, and the sinks through a logarithm)
        return out, lse, np.zeros_like(out), \
            2.0 ** -20 + 2.0 ** -22 * np.abs(alive)
    mean, _ = tree_attention(q, k, np.abs(v), parents, scale, softcap, window,
                             sinks)
    n, hq, depth = q.shape
    group = hq // k.shape[1]
    size = np.stack([np.abs(q[:, h]) @ np.abs(k[:, h // group]).T
                     for h in range(hq)], 1).max(-1) * abs(scale)   # [n, hq]
    d = 2.0 ** -24 * ((depth + 8) * size + 32 * softcap)
    share = np.expm1(2 * d)[..., None] + eps / 2 + 2.0 ** -23 * len(k) + \
        2.0 ** -18
    tiny = len(k) * 2.0 ** -36 * np.abs(v).max() + 2.0 ** -24
    tol = mean * share * (1 + eps) + np.abs(out) * eps / 2 + tiny
    return out, lse, tol, d.T + 2.0 ** -20 + 2.0 ** -22 * np.abs(alive) + \
        2.0 ** -24 * len(k)


def borders(parents, ctx, n_keys, window):
    """Keys at which a row could be lost: the draft's, the last before it,
    those beside every 64th and beside every row's window."""
    n = len(parents)
    seen = tree_mask(parents, ctx, n_keys, window).any(0)
    at = set(range(max(ctx - 2, 0), n_keys))
    start = int(np.argmax(seen)) // 64 * 64 if window >= 0 else 0
    for j in range(start, n_keys, 64):
        at |= {j - 1, j, j + 1}
    if window >= 0:
        at |= {ctx + d - window + e for d in range(min(n, 12))
               for e in (-1, 0)}
    return [j for j in sorted(at) if 0 <= j < n_keys]
