"""Pins of the oracle's norm, group-scaled 4-bit weights and experts' products: hand-worked
values, identities of the definitions, and planted mistakes that the comparisons catch."""
import numpy as np
import pytest

from oracle import experts, group4, norm
from oracle import numerics as onum


def f16(v):
    return np.asarray(v, dtype=np.float32).astype(np.float16)


def test_norm_by_hand():
    # mean of squares of (3, 4, 0, 0) is 25 / 4: rstd = 2 / 5
    h, v = norm.rows(f16([[3, 4, 0, 0]]), "fp16", np.array([1, 2, 3, 4], np.float32), 0.0)
    assert np.array_equal(h, f16([[3, 4, 0, 0]]))
    r = np.float32(0.4)
    assert np.array_equal(v, np.array([[np.float32(3) * r, np.float32(4) * r * np.float32(2), 0, 0]], np.float32))
    codes, scales = norm.quant(v, 8)
    assert codes.tolist() == [[48, 127, 0, 0]] and scales[0] == np.float32(np.float32(3.2) / np.float32(127))


def test_norm_of_the_rounded_sum():
    """The norm is that of the sum as kept in 16 bits: 1 + 2^-12 rounds to 1 in fp16."""
    x, r = f16([[1.0, 1.0]]), f16([[2.0 ** -12, 0.0]])
    h, v = norm.rows(x, "fp16", None, 0.0, r)
    assert np.array_equal(h, x) and np.array_equal(v, np.ones((1, 2), np.float32))


def test_norm_is_scale_free_without_eps():
    rng = np.random.default_rng(1)
    x = f16(rng.standard_normal((4, 64)))
    a = norm.rows(x, "fp16", None, 0.0)[1]
    b = norm.rows(f16(x.astype(np.float32) * 4), "fp16", None, 0.0)[1]
    assert np.array_equal(a, b)  # powers of two are exact throughout


def test_norm_partitions():
    v = np.array([[1.0, -8.0, 2.0, 0.5] + [0.0] * 60], np.float32)
    codes, scales = norm.quant(v, 8, np.array([1]))
    assert codes.shape == (1, 128) and codes[0, 1] == 0 and codes[0, 64] == -127
    assert scales[0, 0] == np.float32(2.0) / np.float32(127) and scales[0, 1] == np.float32(8.0) / np.float32(127)


def test_group_packing_by_hand():
    w = np.zeros((1, 64), np.float32)
    w[0, :4] = [7.0, -3.5, 3.6, -7.0]
    c, packed, s = group4.pack(f16(w), "fp16", 32)
    assert s.astype(np.float32).tolist() == [[1.0, 0.0]]
    assert c[0, :4].tolist() == [7, -4, 4, -7] and not c[0, 4:].any()  # -3.5 is a tie: to even
    assert packed[0, 0] == (7 | (12 << 4)) and np.array_equal(group4.unpack(packed), c)


def test_group_product_is_that_of_the_decoded_weights():
    rng = np.random.default_rng(2)
    w = f16(rng.standard_normal((5, 128)) * 0.1)
    x = f16(rng.standard_normal((3, 128)))
    c, packed, s = group4.pack(w, "fp16", 64)
    y, bound = group4.exact(x, "fp16", packed, s, 64)
    dec = c.astype(np.float64) * np.repeat(s.astype(np.float64), 64, axis=1)
    assert np.allclose(y, x.astype(np.float64) @ dec.T, rtol=1e-14)
    # a weight is off by at most half a step of its group, and a step's rounding to 16 bits
    step = np.repeat(s.astype(np.float64), 64, axis=1)
    assert np.all(np.abs(dec - w.astype(np.float64)) <= 0.5 * step + 7 * step * np.finfo(np.float16).eps)
    # one wrong code is far outside the bound
    bad = packed.copy()
    bad[2, 7] ^= 1
    assert np.max(np.abs(group4.exact(x, "fp16", bad, s, 64)[0] - y) - bound) > 0


def test_nibbles():
    p = np.arange(256, dtype=np.uint8).reshape(1, -1)
    u = group4.unpack(p)[0]
    assert u.min() == -8 and u.max() == 7
    assert u[2 * 0x8F] == -1 and u[2 * 0x8F + 1] == -8


def test_experts_rows():
    a = np.array([[1.0], [2.0], [3.0]])
    w = [np.array([[10.0]]), np.array([[100.0]])]
    y = experts.apply([0, 2, 2, 4], [2, 0, -1, 1], 5, 1, lambda e, i: a[i] * (w + [np.array([[7.0]])])[e])
    assert y[:, 0].tolist()[:4] == [30.0, 10.0, 0.0, 14.0] and np.isnan(y[4, 0])


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_a_wrong_row_is_seen(dt):
    """The comparison of the experts' tests is by bits: a row of another expert differs."""
    rng = np.random.default_rng(3)
    x = onum.from_f32(rng.standard_normal((4, 64)).astype(np.float32), dt)
    w = onum.from_f32(rng.standard_normal((2, 8, 64)).astype(np.float32), dt)
    f = lambda e, i: onum.to_f32(x[i], dt).astype(np.float64) @ onum.to_f32(w[e], dt).astype(np.float64).T  # noqa: E731
    good = experts.apply([0, 2, 4], None, 4, 8, f)
    bad = experts.apply([0, 3, 4], None, 4, 8, f)
    assert np.array_equal(good[[0, 1, 3]], bad[[0, 1, 3]]) and not np.array_equal(good[2], bad[2])
