"""Pins of the oracle's operators between the layers of a block: hand-worked values, identities
of the definitions, and planted mistakes that the comparisons catch."""
import numpy as np

from oracle import gated, lowrank, norm, router
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


def test_routing_by_hand():
    x = np.array([[0.0, 2.0, 1.0, 2.0], [-np.inf, 5.0, -np.inf, -np.inf], [-np.inf] * 4, [1.0, np.nan, 0.0, 0.0]])
    off, rows, w, ch, place = router.route(x, 2)
    assert ch.tolist() == [[1, 3], [1, -1], [-1, -1], [-1, -1]]  # the tie goes to the lower index
    assert off.tolist() == [0, 0, 2, 2, 3] and rows.tolist() == [0, 1, 0] + [-1] * 5
    assert place.tolist() == [[0, 2], [1, -1], [-1, -1], [-1, -1]]
    assert w[:3].tolist() == [[0.5, 0.5], [1.0, 0.0], [0.0, 0.0]] and np.isnan(w[3]).all()
    p = np.exp([0.0, 2.0, 1.0, 2.0])
    assert np.allclose(router.route(x, 2, renorm=False, scale=2.0)[2][0], 2 * p[1] / p.sum(), rtol=1e-15)


def test_a_bias_moves_the_choice_and_not_the_weight():
    x = np.array([[0.0, 1.0, 2.0]])
    ch, w = router.choose(x[0], 1, "sigmoid", bias=[0.9, 0.0, -0.1])
    assert ch == [0] and w == [1.0]
    ch, w = router.choose(x[0], 1, "sigmoid", bias=[0.9, 0.0, -0.1], renorm=False)
    assert w == [0.5]
    assert router.choose(x[0], 3, "sigmoid", bias=[0.0, -np.inf, 0.0])[0] == [2, 0, -1]


def test_groups_by_one_and_by_two():
    x = np.log(np.array([0.30, 0.02, 0.20, 0.18, 0.25, 0.05]))
    assert router.choose(x, 2, groups=3, keep=1)[0] == [0, 1]  # the best single expert is in group 0
    assert router.choose(x, 2, groups=3, keep=1, best=2)[0] == [2, 3]  # the best pair in group 1
    assert router.choose(x, 3, groups=3, keep=2, best=2)[0] == [0, 2, 3]
    # the pairs' sums: 0.32, 0.38, 0.30; with the third group closed but for one expert still third
    x[4] = -np.inf
    assert router.choose(x, 3, groups=3, keep=3, best=2)[0] == [0, 2, 3]


def test_choice_by_the_scores_where_p_rounds_to_one():
    assert router.choose([40.0, 50.0, 45.0], 2, "sigmoid")[0] == [1, 2]
    assert router.choose([-2000.0, 0.0, -1500.0], 2)[0] == [1, 2]


def test_routing_mistakes_are_caught():
    rng = np.random.default_rng(6)
    x = rng.standard_normal((9, 8))
    b = 0.3 * rng.standard_normal(8)
    right = router.route(x, 3, bias=b, groups=4, keep=2, best=2)
    for how in (dict(), dict(bias=b), dict(bias=b, groups=4, keep=2), dict(bias=b, groups=2, keep=1, best=2),
                dict(bias=-b, groups=4, keep=2, best=2), dict(bias=b, groups=4, keep=2, best=2, score="sigmoid")):
        wrong = router.route(x, 3, **how)
        assert not (np.array_equal(right[3], wrong[3]) and np.array_equal(right[2], wrong[2]))


def test_combining_by_hand():
    y = np.array([[1, 2], [10, 20], [np.nan, np.nan]], np.float32)
    place = np.array([[1, 0], [-1, 0], [-1, -1], [1, 5]], np.int32)
    w = np.array([[0.5, 2], [0, 1], [0, 0], [1, np.nan]], np.float32)
    v = router.combine(y, place, w)
    assert v[:3].tolist() == [[7, 14], [1, 2], [0, 0]] and np.isnan(v[3]).all()
    res = np.ones((4, 2), np.float32)
    v = router.combine(y, place, w, res, np.array([[2, -1], [0, 0]], np.float32), np.array([0, 0, 1, 2]))
    assert v.tolist() == [[15, -13], [3, -1], [1, 1], [1, 1]]


def test_a_product_over_experts_and_back_is_the_weighted_sum_of_its_experts():
    rng = np.random.default_rng(7)
    x, wt = rng.standard_normal((6, 4)).astype(np.float32), rng.standard_normal((5, 3, 4)).astype(np.float32)
    off, rows, w, ch, place = router.route(rng.standard_normal((6, 5)), 2)
    y = np.zeros((12, 3), np.float32)
    for e in range(5):
        y[off[e]:off[e + 1]] = x[rows[off[e]:off[e + 1]]] @ wt[e].T
    v = router.combine(y, place, w.astype(np.float32))
    for t in range(6):
        assert np.allclose(v[t], sum(w[t, j] * (wt[ch[t, j]] @ x[t]) for j in range(2)), rtol=1e-5, atol=1e-6)


def test_adapters_by_hand():
    x = np.array([[1.0, 2.0], [3.0, 4.0], [5.0, 6.0]])
    down = np.array([[[1.0, 0.0]], [[0.0, 1.0]]])
    up = np.array([[[1.0], [10.0]], [[2.0], [-1.0]]])
    delta, bound = lowrank.exact(x, down, up, [1, -1, 0], [2.0, 0.5])
    assert delta.tolist() == [[2.0, -1.0], [0.0, 0.0], [10.0, 100.0]]
    assert (bound[1] == 0).all() and (bound[[0, 2]] > 0).all() and (bound < 1e-2).all()


def test_adapters_equal_the_merged_weights():
    """x . (W + s up . down)^T is the projection with the adapter's product merged into its weights."""
    rng = np.random.default_rng(8)
    x, w = rng.standard_normal((5, 16)), rng.standard_normal((7, 16))
    down, up, s = rng.standard_normal((3, 4, 16)), rng.standard_normal((3, 7, 4)), np.array([0.5, 2.0, -1.0])
    index = np.array([0, 2, 3, 1, 0])
    delta, _ = lowrank.exact(x, down, up, index, s)
    for i, a in enumerate(index):
        merged = w if a > 2 else w + s[a] * up[a] @ down[a]
        assert np.allclose(x[i] @ w.T + delta[i], x[i] @ merged.T, rtol=1e-12, atol=1e-12)


def test_adapter_mistakes_are_outside_the_bound():
    rng = np.random.default_rng(9)
    x, down, up = rng.standard_normal((6, 64)), rng.standard_normal((3, 8, 64)) / 8, rng.standard_normal((3, 20, 8))
    index, s = np.array([0, 1, 2, 0, 1, 2]), np.array([0.5, 1.5, 1.0])
    for dt in ("bf16", "fp16"):
        d, b = lowrank.exact(x, down, up, index, s, dt)
        t16 = np.stack([x[i] @ down[a].T for i, a in enumerate(index)]).astype(np.float16).astype(np.float64)
        wrong = [lowrank.exact(x, down, up, (index + 1) % 3, s, dt)[0], lowrank.exact(x, down, up, index, None, dt)[0],
                 np.stack([s[a] * t16[i] @ up[a].T for i, a in enumerate(index)])]  # t rounded once, to 16 bits
        for w in wrong:
            assert (np.abs(w - d) > b).any()
