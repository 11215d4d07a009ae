"""Pins of the attention oracle (CPU): closed forms of the rotation, the append
and the softmax."""

import numpy as np
import pytest

from oracle import attention as A


def test_rotation_is_a_complex_product_and_keeps_lengths():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((3, 48))
    ang = rng.uniform(0, 6, 16)
    for inter in (False, True):
        y = A.rotate(x, np.cos(ang), np.sin(ang), inter)
        a, b = (x[:, 0:32:2], x[:, 1:32:2]) if inter else (x[:, :16], x[:, 16:32])
        z = (a + 1j * b) * np.exp(1j * ang)
        u, w = (y[:, 0:32:2], y[:, 1:32:2]) if inter else (y[:, :16], y[:, 16:32])
        np.testing.assert_allclose(u + 1j * w, z, rtol=1e-14, atol=1e-14)
        np.testing.assert_array_equal(y[:, 32:], x[:, 32:])


def test_rotated_products_depend_on_the_distance_alone():
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((1, 32)), rng.standard_normal((1, 32))
    freq = 10000.0 ** (-np.arange(16) / 16)

    def dot(p, r):
        a = A.rotate(q, np.cos(p * freq), np.sin(p * freq), False)
        b = A.rotate(k, np.cos(r * freq), np.sin(r * freq), False)
        return float((a * b).sum())

    assert dot(100, 93) == pytest.approx(dot(1007, 1000), rel=1e-9)


def test_append_writes_slots_and_skips_padding():
    kc, vc = np.zeros((2, 64, 1, 16)), np.zeros((2, 64, 1, 16))
    k = np.arange(48, dtype=float).reshape(3, 1, 16) + 1
    A.append(k, -k, [65, -1, 128], kc, vc)
    np.testing.assert_array_equal(kc[1, 1], k[0])
    np.testing.assert_array_equal(vc[1, 1], -k[0])
    assert np.count_nonzero(kc) == 16 and np.count_nonzero(vc) == 16


def test_equal_scores_average_and_one_key_is_copied():
    rng = np.random.default_rng(2)
    kc, vc = np.zeros((2, 64, 2, 16)), rng.standard_normal((2, 64, 2, 16))
    q = rng.standard_normal((4, 16))
    keys = [(1, t) for t in range(10)]
    out, lse, _, _ = A.attend(q, kc, vc, keys, 0.3)
    for h in range(4):
        np.testing.assert_allclose(out[h], vc[1, :10, h // 2].mean(0), rtol=1e-13)
    np.testing.assert_allclose(lse, np.log(10))
    out, lse, _, _ = A.attend(q, rng.standard_normal((2, 64, 2, 16)), vc, [(0, 5)], 0.3)
    np.testing.assert_allclose(out, vc[0, 5].repeat(2, 0), rtol=1e-13)


def test_weights_are_the_softmax_of_the_scaled_products():
    kc = np.zeros((1, 64, 1, 16))
    vc = np.zeros((1, 64, 1, 16))
    kc[0, 0, 0, 0], kc[0, 1, 0, 0] = np.log(3.0), 0.0
    vc[0, 0, 0, 0] = 1.0
    q = np.zeros((1, 16))
    q[0, 0] = 2.0
    out, lse, _, _ = A.attend(q, kc, vc, [(0, 0), (0, 1)], 0.5)
    assert out[0, 0] == pytest.approx(0.75) and lse[0] == pytest.approx(np.log(4.0))


def test_visible_keys():
    starts, ends, table = [0, 1, 3], [65, 1, 2, 9], [[4, 5], [6, 7]]
    assert A.visible(0, starts, ends, table)[63:] == [(4, 63), (5, 0)]
    assert A.visible(2, starts, ends, table) == [(6, 0), (6, 1)]
    assert A.visible(3, starts, ends, table, [9], 3) == []                      # a padding row
    assert A.visible(1, starts, ends, table, [9], 2) == [(9, 0), (9, 1), (6, 0)]
    topk = [[64, -1, 0, 65], [0, 1, -1, -1], [-1] * 4, [0] * 4]
    assert A.visible(0, starts, ends, table, topk=topk) == [(5, 0), (4, 0)]
    assert A.visible(1, starts, ends, table, topk=topk) == [(6, 0)]
    assert A.visible(2, starts, ends, table, topk=topk) == []
