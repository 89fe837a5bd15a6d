"""Pins of the oracle's operators between the layers of a block: hand-worked values, identities
of the definitions, and planted mistakes that the comparisons catch."""
import numpy as np

from oracle import gated, norm
from oracle import numerics as onum


def f16(v):
    return np.asarray(v, dtype=np.float32).astype(np.float16)


def test_layer_norm_by_hand():
    # mean 2, deviations -1 and 1, variance 1 (eps 0)
    s, v = gated.rows(None, f16([[1, 3, 1, 3]]), "fp16", "layer", eps=0.0)
    assert np.array_equal(s, f16([[1, 3, 1, 3]])) and v.tolist() == [[-1.0, 1.0, -1.0, 1.0]]


def test_gate_and_residual_scale_by_hand():
    # the branch (2, 2) has rms 2, so its norm is (1, 1); gate (3, -1), residual scale 1/2
    g = np.array([[3.0, -1.0]], np.float32)
    s, v = gated.rows(f16([[2, 2]]), f16([[1, 1]]), "fp16", "rms", post="rms", alpha=0.5, gate=g, eps=0.0)
    assert s.astype(np.float32).tolist() == [[2.5, 0.5]]
    r = np.float32(1.0 / np.sqrt((2.5 ** 2 + 0.5 ** 2) / 2))
    assert np.array_equal(v, np.array([[np.float32(2.5) * r, np.float32(0.5) * r]]))


def test_scale_and_shift_by_set():
    h = f16([[1, -1], [1, -1], [1, -1], [1, -1]])
    c, d = np.array([[0, 0], [1, 1]], np.float32), np.array([[0, 0], [0.5, 0]], np.float32)
    _, even = gated.rows(None, h, "fp16", scale=c, shift=d, eps=0.0)
    assert even.tolist() == [[1, -1], [1, -1], [2.5, -2], [2.5, -2]]
    _, by = gated.rows(None, h, "fp16", scale=c, shift=d, index=[1, 0, 7, -1], eps=0.0)
    assert by.tolist() == [[2.5, -2], [1, -1], [1, -1], [1, -1]]


def test_a_row_outside_the_sets_has_no_branch():
    y, h = f16([[np.nan, np.inf], [1, 1]]), f16([[1, 2], [1, 2]])
    s, v = gated.rows(y, h, "fp16", gate=np.ones((1, 2), np.float32), index=[-1, 0])
    assert s.astype(np.float32).tolist() == [[1, 2], [2, 3]] and np.isfinite(v).all()


def test_without_gate_and_mean_it_is_the_norm_of_the_sum():
    rng = np.random.default_rng(3)
    y, h = f16(rng.standard_normal((5, 96))), f16(rng.standard_normal((5, 96)))
    w = (1 + 0.1 * rng.standard_normal(96)).astype(np.float32)
    for dt, a, b in (("fp16", y, h), ("bf16", onum.from_f32(y.astype(np.float32), "bf16"), onum.from_f32(h.astype(np.float32), "bf16"))):
        s, v = gated.rows(a, b, dt, "rms", w, 1e-6)
        s2, v2 = norm.rows(a, dt, w, 1e-6, b)
        assert np.array_equal(s, s2) and np.array_equal(v, v2)


def test_one_pass_variance_keeps_its_digits():
    """The kernel's variance, sum x^2 / K - mean^2 in float64, against the two passes here: a mean a
    thousand times the deviation."""
    rng = np.random.default_rng(4)
    x = f16(4000 + 4 * rng.integers(-1, 2, (3, 4096))).astype(np.float64)
    one = (x * x).sum(1) / 4096 - (x.sum(1) / 4096) ** 2
    two = ((x - x.mean(1, keepdims=True)) ** 2).sum(1) / 4096
    assert np.all(np.abs(one - two) <= 4096 * 2.0 ** -53 * (x * x).mean(1))
    assert np.array_equal((1 / np.sqrt(one)).astype(np.float32), (1 / np.sqrt(two)).astype(np.float32))


def test_planted_mistakes_are_caught():
    rng = np.random.default_rng(5)
    y, h = f16(rng.standard_normal((4, 64))), f16(2 + rng.standard_normal((4, 64)))
    g = (1 + 0.3 * rng.standard_normal((2, 64))).astype(np.float32)
    s, v = gated.rows(y, h, "fp16", "layer", post="rms", gate=g, scale=g, shift=g)
    wrong = [
        gated.rows(y, h, "fp16", "rms", post="rms", gate=g, scale=g, shift=g),  # no mean
        gated.rows(y, h, "fp16", "layer", gate=g, scale=g, shift=g),  # no post norm
        gated.rows(y, h, "fp16", "layer", post="rms", gate=g[::-1], scale=g, shift=g),  # another set
        gated.rows(y, h, "fp16", "layer", post="rms", gate=g, scale=g - 1, shift=g),  # scale for 1 + scale
        gated.rows(h, y, "fp16", "layer", post="rms", gate=g, scale=g, shift=g),  # operands changed over
    ]
    for ws, wv in wrong:
        assert not (np.array_equal(ws, s) and np.array_equal(wv, v))
