"""What pins the oracles of the 4-bit cache and of norms and rotations."""
import numpy as np
import pytest
import torch

from oracle.fp4 import (dequantize_fp4_ref, e2m1_decode, e2m1_encode,
                        pack_codes, quantize_fp4_ref, unpack_codes)
from oracle.fp8 import e4m3_decode
from oracle.rope import axis_of_pair, make_table, norm_rope_ref, pairwise_sum


def test_e2m1_codes_by_definition():
    for c in range(16):
        e, m = (c >> 1) & 3, c & 1
        v = m * 0.5 if e == 0 else (1 + m / 2) * 2.0 ** (e - 1)
        assert e2m1_decode(c) == (-v if c & 8 else v)
    assert np.array_equal(e2m1_encode(e2m1_decode(np.arange(16))),
                          np.arange(16))


def test_e2m1_rounding_by_hand():
    # midpoints go to the even code; beyond 6 saturates
    x = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, 0.26, 0.74, 5.01, -0.25,
         -5.0, np.inf]
    want = [0, 1, 1, 2, 2, 4, 4, 6, 0.5, 0.5, 6, 0, -4, 6]
    assert np.array_equal(e2m1_decode(e2m1_encode(x)), want)


def test_e2m1_is_nearest():
    x = np.random.default_rng(0).uniform(-7, 7, 4000)
    grid = e2m1_decode(np.arange(16))
    best = np.abs(x[:, None] - grid).min(1)
    assert np.array_equal(np.abs(x - e2m1_decode(e2m1_encode(x))), best)


def test_packing_order():
    codes = np.arange(16, dtype=np.uint8)
    p = pack_codes(codes)
    assert p[0] == 0x10 and p[7] == 0xFE
    assert np.array_equal(unpack_codes(p), codes)


@pytest.mark.parametrize("scale", [1.0, 0.0021, 0.25])
def test_quantization_error_bound(scale):
    """Half the widest code step (1, between 4 and 6) of the block scale,
    plus the scale's own rounding (2^-4 relative) of the largest value."""
    x = np.random.default_rng(1).standard_normal((50, 128)).astype(np.float32)
    packed, sf = quantize_fp4_ref(x, scale)
    y = dequantize_fp4_ref(packed, sf, scale)
    top = np.repeat(np.abs(x).reshape(50, 8, 16).max(-1), 16, axis=-1)
    assert np.all(np.abs(x - y) <= top * (1 / 6 * (1 + 2 ** -4) + 2 ** -4))


def test_quantization_special_groups():
    x = np.zeros((4, 16), np.float32)
    x[1, 3] = np.nan
    x[2, 5] = -np.inf
    x[2, 6] = 2.0
    x[3, 0] = 1e-30
    packed, sf = quantize_fp4_ref(x, 1.0)
    y = dequantize_fp4_ref(packed, sf)
    assert not y[0].any() and np.isnan(y[1]).all()
    assert y[2, 5] == -2688.0 and np.isnan(e4m3_decode(sf[1])).all()
    assert not y[3].any()


def test_rotation_is_a_rotation():
    """Against complex multiplication, and norms of pairs are kept."""
    rng = np.random.default_rng(2)
    x = rng.standard_normal((7, 3, 32))
    pos = rng.integers(0, 90, 7)
    table = make_table(90, 24)
    y = norm_rope_ref(x, None, pos, table, neox=False)
    z = x[..., 0:24:2] + 1j * x[..., 1:24:2]
    freq = 10000.0 ** (-np.arange(0, 24, 2) / 24)
    z = z * np.exp(1j * pos[:, None] * freq)[:, None]
    assert np.abs(y[..., 0:24:2] - z.real).max() < 1e-12
    assert np.abs(y[..., 1:24:2] - z.imag).max() < 1e-12
    assert np.array_equal(y[..., 24:], x[..., 24:])
    w = norm_rope_ref(x, None, pos, table, neox=True)
    perm = np.r_[0:24:2, 1:24:2]
    xp = x.copy()
    xp[..., 0:24:2], xp[..., 1:24:2] = x[..., :12], x[..., 12:24]
    assert np.abs(norm_rope_ref(xp, None, pos, table, neox=False)[..., perm] -
                  w[..., :24]).max() < 1e-12


def test_relative_positions_only():
    """q at p and k at j after rotation: the product depends on p - j."""
    rng = np.random.default_rng(3)
    q, k = rng.standard_normal((2, 1, 1, 64))
    table = make_table(500, 64)

    def dot(p, j):
        a = norm_rope_ref(q, None, [p], table)
        return (a * norm_rope_ref(k, None, [j], table)).sum()
    assert abs(dot(120, 20) - dot(420, 320)) < 1e-10


def test_norm_against_torch():
    x = torch.randn(5, 2, 80, dtype=torch.float64)
    w = torch.randn(80, dtype=torch.float64)
    got = norm_rope_ref(x.numpy(), w.numpy(), [0] * 5, make_table(1, 16))
    want = torch.nn.functional.rms_norm(x, (80,), w, float(np.float32(1e-6)))
    assert np.abs(got - want.numpy()).max() < 1e-12


def test_axes():
    assert list(axis_of_pair(6, [2, 3, 1], False)) == [0, 0, 1, 1, 1, 2]
    assert list(axis_of_pair(6, [2, 2, 2], True)) == [0, 1, 2, 0, 1, 2]
    assert list(axis_of_pair(8, [4, 2, 2], True)) == [0, 1, 2, 0, 1, 2, 0, 0]
    # equal positions on every axis are plain positions
    x = np.random.default_rng(4).standard_normal((3, 1, 16))
    t = make_table(50, 16)
    one = norm_rope_ref(x, None, [4, 9, 30], t)
    many = norm_rope_ref(x, None, np.tile([4, 9, 30], (3, 1)), t,
                         sections=[2, 3, 3], interleaved=True)
    assert np.array_equal(one, many)


def test_pairwise_sum_pads():
    x = np.arange(1.0, 12.0)
    assert pairwise_sum(x)[0] == 66.0
