"""The 4-bit cache's oracle, pinned on the CPU: the layout by hand, the quantiser against a search of the codebook."""

import numpy as np
import pytest

from oracle import fp4_cache as F
from oracle.codecs import E2M1_TABLE, E4M3_TABLE


def test_layout_by_hand():
    """One token of one head of 32 columns, every byte in its place."""
    cache = np.zeros((2, 1, F.section_bytes(32)), dtype=np.uint8)
    assert cache.shape[2] == 64 * (16 + 16 + 8)
    k = np.zeros((1, 1, 32))
    k[0, 0, :4] = [6, -3, 0.5, 1]           # scale 1: codes 7, 13, 1, 2
    v = np.zeros((1, 1, 32))
    v[0, 0, 16:18] = [12, -2]               # scale 2 of the second block: codes 7, 10
    F.append(k, v, [64 + 5], cache, 32)
    want = np.zeros_like(cache)
    want[1, 0, 5 * 16: 5 * 16 + 2] = [0xD7, 0x21]
    want[1, 0, 64 * 16 + 5 * 16 + 8] = 0xA7
    scales = 2 * 64 * 16 + 5 * 8
    want[1, 0, scales] = 0x38               # E4M3 1
    want[1, 0, scales + 4 + 1] = 0x40       # E4M3 2
    np.testing.assert_array_equal(cache, want)
    keys, values = F.decode(cache, 32)
    np.testing.assert_array_equal(keys[1, 5, 0, :4], [6, -3, 0.5, 1])
    np.testing.assert_array_equal(values[1, 5, 0, 16:18], [12, -2])


@pytest.mark.parametrize("g", [1.0, 0.25, 0.37, 1e-9])
def test_quantiser_against_the_codebook(g):
    """The scale is the E4M3 value nearest to amax / (6 g), every code the E2M1 value nearest to x / (s g)."""
    rng = np.random.default_rng(1)
    x = (rng.standard_normal((300, 16)) * np.exp(rng.uniform(-8, 8, (300, 1))) * g).astype(np.float32)
    codes, scales = F.quantise(x, g)
    finite = E4M3_TABLE[np.isfinite(E4M3_TABLE) & (E4M3_TABLE >= 0)]
    g = float(np.float32(g))
    stood = F.values(codes, scales, g)
    for row, s, got in zip(x.astype(np.float64), scales[:, 0], stood):
        ratio = np.abs(row).max() / (6 * g)
        assert abs(E4M3_TABLE[s] - ratio) <= np.abs(finite - ratio).min() + 1e-6 * ratio
        if E4M3_TABLE[s] == 0:
            assert not got.any()
            continue
        y = row / (E4M3_TABLE[s] * g)
        best = np.abs(E2M1_TABLE[None, :] - y[:, None]).min(axis=1)
        assert (np.abs(got / (E4M3_TABLE[s] * g) - y) <= best + 1e-6 * np.maximum(1, np.abs(y))).all()


def test_special_blocks():
    x = np.zeros((5, 16), dtype=np.float32)
    x[1, 3] = np.nan
    x[2, 4], x[2, 5] = np.inf, 1.0
    x[3] = 1e-6                             # under half of the smallest scale
    x[4, 0], x[4, 1] = 1e9, -1e9
    codes, scales = F.quantise(x, 1.0)
    v = F.values(codes, scales, 1.0)
    assert not v[0].any() and np.isnan(v[1]).all() and not v[3].any()
    assert v[2, 4] == 2688 and v[2, 5] == 0 and v[4, 0] == 2688 and v[4, 1] == -2688


def test_ties_go_to_even_codes():
    x = np.array([[6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5, 0]], dtype=np.float32)
    v = F.values(*F.quantise(x, 1.0), 1.0)
    np.testing.assert_array_equal(v[0], [6, 0, 1, 1, 2, 2, 4, 4, 0, -1, -1, -2, -2, -4, -4, 0])


def test_quotient_by_reciprocal_and_one_correction():
    """x / d from q0 = x RN(1 / d) and one correction by its remainder is the correctly rounded quotient, next to the
    borders between codes too (the remainder of a fused multiply-add is exact: emulated in 64 bits)."""
    rng = np.random.default_rng(2)
    f32 = np.float32
    s = E4M3_TABLE[1:0x7F].astype(f32)
    for g in (f32(1), f32(0.37), f32(1.3e-7), f32(2) ** 60):
        d = np.repeat(s * g, 400)
        border = rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 1.0, 7.9], d.size)
        x = (d.astype(np.float64) * border).astype(f32)
        x = np.where(rng.random(d.size) < 0.7, np.nextafter(x, rng.choice([-1, 1], d.size).astype(f32) * f32(np.inf)), x)
        inv = f32(1) / d
        q0 = x * inv
        r = (x.astype(np.float64) - q0.astype(np.float64) * d.astype(np.float64)).astype(f32)
        # q0 + r inv in 64 bits: the product is exact, the sum is off by 2^-53 of it, far under a half step of FP32
        # unless the quotient is that near to one, which no x / d with 24-bit x and d is
        y = (q0.astype(np.float64) + r.astype(np.float64) * inv.astype(np.float64)).astype(f32)
        np.testing.assert_array_equal(y, x / d)


def test_rotation_is_in_fp32():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((2, 3, 32)).astype(np.float32)
    ang = rng.uniform(0, 6, (2, 8))
    c, s = np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)
    for inter in (False, True):
        y = F.rotate(x, c, s, inter)
        a, b = (0, 1) if inter else (0, 8)
        np.testing.assert_array_equal(y[:, :, a], x[:, :, a] * c[:, :1] - x[:, :, b] * s[:, :1])
        np.testing.assert_array_equal(y[..., 16:], x[..., 16:])
