"""Head norms and rotary positions: oracle.

TEST INFRASTRUCTURE ONLY (see oracle/__init__.py).

``norm_rope_ref`` is the formula; evaluated in float64 it is the reference,
and in float32 (each operation rounded, the sum of squares pairwise) it is
the operator's definition before its last rounding.
"""
from __future__ import annotations

import numpy as np


def axis_of_pair(half, sections, interleaved):
    """Axis whose position rotates pair 0 .. half - 1."""
    if not sections:
        return np.zeros(half, np.int64)
    if not interleaved:
        return np.repeat(np.arange(len(sections)), sections)
    i = np.arange(half)
    a = i % len(sections)
    return np.where(i < len(sections) * np.asarray(sections)[a], a, 0)


def pairwise_sum(x):
    """Sum over the last axis, neighbours first (padded to a power of 2)."""
    n = 1
    while n < x.shape[-1]:
        n *= 2
    pad = np.zeros(x.shape[:-1] + (n - x.shape[-1],), x.dtype)
    x = np.concatenate([x, pad], -1)
    while x.shape[-1] > 1:
        x = x[..., 0::2] + x[..., 1::2]
    return x


def norm_rope_ref(x, weight, positions, table, *, eps=1e-6, offset=0.0,
                  neox=True, sections=None, interleaved=False,
                  dtype=np.float64):
    """Rows x [T, H, D] -> [T, H, D] in dtype, unrounded.

    weight [D] or None; positions [T] or [axes, T]; table [P, rot]."""
    f = dtype
    x = np.asarray(x).astype(f)
    D = x.shape[-1]
    rot = table.shape[1]
    half = rot // 2
    if weight is not None:
        ms = pairwise_sum(x * x) / f(D)
        r = f(1) / np.sqrt(ms + f(np.float32(eps)))
        x = x * r * (np.asarray(weight).astype(f) + f(np.float32(offset)))
    pos = np.asarray(positions)
    pos = pos[None] if pos.ndim == 1 else pos
    at = pos[axis_of_pair(half, sections, interleaved)].T      # [T, half]
    i = np.arange(half)
    c = np.asarray(table)[at, i].astype(f)[:, None]
    s = np.asarray(table)[at, half + i].astype(f)[:, None]
    y = x.copy()
    if neox:
        a, b = x[..., :half], x[..., half:rot]
        y[..., :half], y[..., half:rot] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * s, b * c + a * s
    return y


def make_table(positions, rot, base=10000.0):
    """cos | sin of a plain rotary table, float64 [positions, rot]."""
    freq = base ** (-np.arange(0, rot, 2) / rot)
    angle = np.arange(positions)[:, None] * freq
    return np.concatenate([np.cos(angle), np.sin(angle)], -1)
