"""4-bit KV cache (E2M1 codes, E4M3 scales of 16 values): oracle.

TEST INFRASTRUCTURE ONLY (see oracle/__init__.py).

E2M1: 1 sign bit, 2 exponent bits (bias 1), 1 mantissa bit; exponent 0 holds
0 and 0.5; the magnitudes are 0, 0.5, 1, 1.5, 2, 3, 4, 6.  Two codes share a
byte, the lower index in the lower four bits.

The definition of the quantization of 16 values x of a row, each step rounded
to float32 (numpy's float32 arithmetic is IEEE):
  a = max |x|;  block_scale = e4m3(a * fl(1 / fl(6 * scale)))
  code = e2m1(x * fl(1 / fl(block_scale * scale)))   (0 if that scale is 0)
to nearest, ties to even, saturated; a NaN makes the block scale NaN.
"""
from __future__ import annotations

import numpy as np

from .fp8 import e4m3_decode, e4m3_encode

_MAG = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e2m1_decode(codes) -> np.ndarray:
    """float64 values of 4-bit codes (0 .. 15)."""
    c = np.asarray(codes, dtype=np.int64)
    return np.where(c & 8, -1.0, 1.0) * _MAG[c & 7]


def e2m1_encode(x) -> np.ndarray:
    """Nearest E2M1 code, ties to the even code, saturated at +-6."""
    x = np.asarray(x, dtype=np.float64)
    a = np.abs(x)
    hi = np.clip(np.searchsorted(_MAG, a), 1, 7)
    d_lo, d_hi = a - _MAG[hi - 1], _MAG[hi] - a
    up = (d_lo > d_hi) | ((d_lo == d_hi) & (hi % 2 == 0))
    code = np.where(a >= 6.0, 7, np.where(up, hi, hi - 1))
    return (code | np.where(np.signbit(x), 8, 0)).astype(np.uint8)


def pack_codes(codes) -> np.ndarray:
    """[..., D] codes -> [..., D / 2] bytes."""
    c = np.asarray(codes, dtype=np.uint8)
    return (c[..., 0::2] | (c[..., 1::2] << 4)).astype(np.uint8)


def unpack_codes(packed) -> np.ndarray:
    p = np.asarray(packed, dtype=np.uint8)
    return np.stack([p & 15, p >> 4], -1).reshape(
        p.shape[:-1] + (2 * p.shape[-1],))


def quantize_fp4_ref(x, scale):
    """Rows [..., D] of float32 values -> (packed codes [..., D / 2], E4M3
    block scale codes [..., D / 16])."""
    f = np.float32
    x = np.asarray(x, dtype=f)
    scale = f(scale)
    g = x.reshape(x.shape[:-1] + (x.shape[-1] // 16, 16))
    with np.errstate(all="ignore"):
        top = np.abs(g).max(-1)                  # NaN stays
        sf = e4m3_encode(top * (f(1) / (f(6) * scale)))
        step = e4m3_decode(sf).astype(f) * scale
        inv = np.where(step > 0, f(1) / step, f(0)).astype(f)
        y = g * inv[..., None]
    codes = e2m1_encode(np.where(np.isnan(y), 0.0, y)).reshape(x.shape)
    return pack_codes(codes), sf


def dequantize_fp4_ref(packed, sf, scale=1.0) -> np.ndarray:
    """float64 values of a cache's rows."""
    v = e2m1_decode(unpack_codes(packed))
    s = np.repeat(e4m3_decode(sf), 16, axis=-1)
    return v * s * np.float64(np.float32(scale))


def reshape_and_cache_fp4_ref(key, value, key_cache, value_cache, k_sf, v_sf,
                              slot_mapping, k_scale, v_scale):
    """The quantizing cache write, in place (slots < 0 are skipped)."""
    bs = key_cache.shape[1]
    for rows, codes, sf, sc in ((key, key_cache, k_sf, k_scale),
                                (value, value_cache, v_sf, v_scale)):
        packed, s = quantize_fp4_ref(np.asarray(rows)[:len(slot_mapping)], sc)
        for t, slot in enumerate(slot_mapping):
            if slot >= 0:
                codes[slot // bs, slot % bs] = packed[t]
                sf[slot // bs, slot % bs] = s[t]
