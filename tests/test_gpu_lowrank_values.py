"""Low-rank adapters: infinities among their weights, and a float32 output of bfloat16 operands."""
import numpy as np
import pytest
import torch

import gen
from oracle import lowrank as ol
from oracle import numerics as onum

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def vq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_quantized_linear_vq_amd as m
    return m


def f64(t, dt):
    return onum.to_f32(gen.as_numpy_bits(t), dt).astype(np.float64)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("r", [8, 64, 104])
@pytest.mark.parametrize("m", [5, 200, 1100])
def test_an_infinite_weight_of_up_is_an_infinity_of_its_sign(vq, m, r, dt):
    """t times an infinity, whatever the pieces in which t goes on: its own sign where t is not zero, NaN where
    t is zero or two infinities meet, and the other columns as they are."""
    rng = np.random.default_rng([m, r])
    k, n, ad = 64, 70, 3

    def whole(shape, big):
        return rng.integers(-big, big + 1, shape).astype(np.float32)
    x, down = gen.to_storage(whole((m, k), 4), dt), gen.to_storage(whole((ad, r, k), 3), dt)
    u = whole((ad, n, r), 5)
    u[1, 3, 2], u[1, 40, 0], u[1, 69, r - 1] = np.inf, -np.inf, np.inf
    u[2, 10, 1], u[2, 10, 4] = np.inf, -np.inf
    up = gen.to_storage(u, dt)
    index = torch.from_numpy(rng.integers(-1, ad, m).astype(np.int32))
    scales = torch.tensor([1.0, 0.5, 0.3])
    base = torch.from_numpy(whole((m, n), 99))
    x[0] = 0  # t = 0: NaN in those columns
    index[:3] = torch.tensor([1, 1, 2])
    got = vq.vq_lowrank_add(base.to(DEV), x.to(DEV), down.to(DEV), up.to(DEV), index.to(DEV), scales=scales.to(DEV))
    torch.cuda.synchronize()
    with np.errstate(invalid="ignore"):
        delta, bound = ol.exact(f64(x, dt), f64(down, dt), f64(up, dt), index.numpy(), scales.numpy(), dt)
    want, g = base.numpy().astype(np.float64) + delta, got.cpu().numpy().astype(np.float64)
    odd = ~np.isfinite(want)
    assert odd.any() and np.isinf(want).any() and np.isnan(want).any()
    assert np.array_equal(g[odd], want[odd], equal_nan=True)
    off, delta, bound, base = np.abs(g[~odd] - want[~odd]), delta[~odd], bound[~odd], base.numpy()[~odd]
    assert np.all(off <= bound + 2.0 ** -23 * (np.abs(base) + np.abs(delta) + bound))


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("m", [5, 1100])
def test_an_infinite_t_beside_large_ones(vq, m, dt):
    """One infinite t in a row whose others are beyond fp16's range: the infinity's sign, whatever theirs."""
    rng = np.random.default_rng(m)
    k, n, r, ad = 64, 40, 16, 2
    x = gen.to_storage((3e4 * (1 + rng.random((m, k)))).astype(np.float32), dt)
    d = (1 + rng.random((ad, r, k))).astype(np.float32)  # every t far above 65504
    d[1, 3, 5] = np.inf
    u = np.full((ad, n, r), -1.0, np.float32)
    u[:, :, 3] = 1.0
    u[:, ::2] *= -1.0
    down, up = gen.to_storage(d, dt), gen.to_storage(u, dt)
    index = torch.arange(m, dtype=torch.int32) % 3 - 1
    base = torch.zeros(m, n)
    got = vq.vq_lowrank_add(base.to(DEV), x.to(DEV), down.to(DEV), up.to(DEV), index.to(DEV)).cpu().numpy().astype(np.float64)
    delta, bound = ol.exact(f64(x, dt), f64(down, dt), f64(up, dt), index.numpy(), None, dt)
    odd = ~np.isfinite(delta)
    assert np.isinf(delta[index.numpy() == 1]).all() and np.array_equal(got[odd], delta[odd])
    assert np.all(np.abs(got[~odd] - delta[~odd]) <= bound[~odd] + 2.0 ** -23 * (np.abs(delta[~odd]) + bound[~odd]))


@pytest.mark.parametrize("m,n,k,r,adapters", [(1, 96, 512, 64, 1), (40, 130, 256, 16, 4), (64, 70, 4096, 128, 3), (200, 515, 128, 40, 5),
                                              (1100, 129, 192, 128, 6), (1025, 320, 320, 32, 2)])
def test_a_float32_output_of_bfloat16_operands(vq, m, n, k, r, adapters):
    """t goes on in three pieces of 8 bits, which are t: nothing but the float32 sums is lost."""
    rng = np.random.default_rng([m, n, k, r])

    def half(shape, scale):
        return gen.to_storage((scale * rng.standard_normal(shape)).astype(np.float32), "bf16")
    # K of few terms that are not zero, so that the first product's own roundings are few
    x = half((m, k), 1.0)
    x[:, 3:] = 0
    down, up = half((adapters, r, k), 1.0), half((adapters, n, r), r ** -0.5)
    up[:, :, 1:] = 0  # one term: t's pieces times one weight, and a rounding of each sum
    index = torch.from_numpy(rng.integers(-1, adapters, m).astype(np.int32))
    index[0] = 0
    base = torch.zeros(m, n)
    got = vq.vq_lowrank_add(base.to(DEV), x.to(DEV), down.to(DEV), up.to(DEV), index.to(DEV))
    torch.cuda.synchronize()
    xd, dd, ud = f64(x, "bf16"), f64(down, "bf16"), f64(up, "bf16")
    delta, _ = ol.exact(xd, dd, ud, index.numpy(), None, "bf16")
    bound = np.zeros((m, n))
    for a in range(adapters):
        at = np.nonzero(index.numpy() == a)[0]
        ta = np.abs(xd[at]) @ np.abs(dd[a]).T  # three products, two additions that round, the zeros' none
        bound[at] = (4 * ta * 2.0 ** -23 + 4 * np.abs(xd[at] @ dd[a].T) * 2.0 ** -23) @ np.abs(ud[a]).T
    assert np.all(np.abs(got.cpu().numpy().astype(np.float64) - delta) <= bound)


@pytest.mark.parametrize("m,n,k,r,adapters", [(3, 33, 128, 24, 2), (64, 100, 1024, 64, 5), (200, 257, 640, 128, 9), (1100, 320, 256, 16, 4)])
def test_a_float32_output_within_the_bound_of_three_pieces(vq, m, n, k, r, adapters):
    rng = np.random.default_rng([m, n, k])

    def half(shape, scale):
        return gen.to_storage((scale * rng.standard_normal(shape)).astype(np.float32), "bf16")
    x, down, up = half((m, k), 1.0), half((adapters, r, k), k ** -0.5), half((adapters, n, r), r ** -0.5)
    index = torch.from_numpy(rng.integers(-1, adapters, m).astype(np.int32))
    scales = torch.from_numpy((0.5 + rng.random(adapters)).astype(np.float32))
    base = torch.from_numpy(rng.standard_normal((m, n)).astype(np.float32))
    got = vq.vq_lowrank_add(base.to(DEV), x.to(DEV), down.to(DEV), up.to(DEV), index.to(DEV), scales=scales.to(DEV)).cpu().numpy()
    delta, bound = ol.exact(f64(x, "bf16"), f64(down, "bf16"), f64(up, "bf16"), index.numpy(), scales.numpy(), "bf16", out="fp32")
    b = base.numpy().astype(np.float64)
    assert np.all(np.abs(got - (b + delta)) <= bound + 2.0 ** -24 * (np.abs(b + delta) + bound))
