"""The group-scaled 4-bit product where a worst-case bound of large sums says little: loud
channels against the codes that they meet, and the largest and infinite values of x."""
import numpy as np
import pytest
import torch

import gen
from oracle import group4
from oracle import numerics as onum

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def vq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_quantized_linear_vq_amd as m
    return m


def pack(c):
    return torch.from_numpy(((c[:, 0::2] & 15) | ((c[:, 1::2] & 15) << 4)).astype(np.uint8)).to(DEV)


@pytest.mark.parametrize("dt,loud", [("bf16", 1e4), ("bf16", 1e5), ("bf16", 2.0 ** 100), ("fp16", 1e4), ("fp16", 5e4)])
@pytest.mark.parametrize("m,group", [(1, 128), (5, 32), (20, 64)])
def test_a_loud_channel_costs_nothing_where_its_code_is_zero(vq, m, group, dt, loud):
    """The other channels keep the accuracy of their own sum: the bound counts |s c x|."""
    n, k = 200, 2048
    rng = np.random.default_rng([m, group])
    c = rng.integers(-8, 8, (n, k))
    c[:, 5] = 0
    c[:, k - 1] = 0
    x = rng.standard_normal((m, k)).astype(np.float32)
    x[:, 5] = loud
    x[:, k - 1] = -loud
    xs = gen.to_storage(x, dt)
    s = gen.to_storage((0.01 + 0.02 * rng.random((n, k // group))).astype(np.float32), dt)
    y = vq.vq_w4_gemv(xs.to(DEV), pack(c), s.to(DEV), torch.float32).cpu().numpy()
    ex, b = group4.exact(gen.as_numpy_bits(xs), dt, pack(c).cpu().numpy(), gen.as_numpy_bits(s), group)
    assert np.all(np.abs(y - ex) <= b), float((np.abs(y - ex) / b).max())


@pytest.mark.parametrize("dt,large", [("bf16", 3e37), ("bf16", 1e38), ("fp16", 65504.0)])
def test_large_finite_rows_have_finite_outputs(vq, dt, large):
    """A group's sum is that of its codes: 3 * 1e38 is finite, and so is 0 * 1e38."""
    n, k = 40, 256
    c = np.ones((n, k), dtype=np.int64)
    c[:, 3], c[:, 200], c[:, 201] = 0, 3, -2
    x = np.ones((2, k), dtype=np.float32)
    x[:, 3] = large
    x[1, 200] = large
    xs = gen.to_storage(x, dt)
    s = gen.to_storage(np.full((n, k // 128), 0.5, dtype=np.float32), dt)
    y = vq.vq_w4_gemv(xs.to(DEV), pack(c), s.to(DEV), torch.float32).cpu().numpy()
    ex, b = group4.exact(gen.as_numpy_bits(xs), dt, pack(c).cpu().numpy(), gen.as_numpy_bits(s), 128)
    assert np.all(np.isfinite(y)) and np.all(np.abs(y - ex) <= b)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_an_infinity_meets_its_code(vq, dt):
    k, n = 128, 16
    c = np.ones((n, k), dtype=np.int64)
    c[:, 9] = np.arange(n) - 8
    x = np.ones((3, k), dtype=np.float32)
    x[1, 9], x[2, 9] = np.inf, -np.inf
    y = vq.vq_w4_gemv(gen.to_storage(x, dt).to(DEV), pack(c), torch.ones((n, 1), dtype=gen.to_storage(x, dt).dtype, device=DEV),
                      torch.float32).cpu().numpy()
    assert np.array_equal(y[0], c.sum(1).astype(np.float32))
    with np.errstate(invalid="ignore"):
        want = np.float32(np.inf) * c[:, 9].astype(np.float32)
    assert np.array_equal(y[1], want, equal_nan=True) and np.array_equal(y[2], -want, equal_nan=True)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_weights_that_are_not_finite(vq, dt, group):
    """Their group has a NaN scale and zero codes, the other groups are as without them, and the
    channel's outputs say so."""
    rng = np.random.default_rng(group)
    n, k = 9, 3 * group
    w = (rng.standard_normal((n, k)) * 0.02).astype(np.float32)
    clean = vq.vq_pack_weights_group(gen.to_storage(w, dt).to(DEV), group)[0].cpu().numpy()
    w[1, 0], w[2, group - 1], w[3, group + 5], w[4, 3 * group - 1] = np.nan, np.inf, -np.inf, np.nan
    w[5, group:2 * group] = np.nan
    w[6, 3], w[6, 4] = np.inf, np.nan
    ws = gen.to_storage(w, dt)
    codes, scales = vq.vq_pack_weights_group(ws.to(DEV), group)
    bad = np.zeros((n, 3), dtype=bool)
    bad[1, 0] = bad[2, 0] = bad[3, 1] = bad[4, 2] = bad[5, 1] = bad[6, 0] = True
    _, packed, s = group4.pack(gen.as_numpy_bits(ws), dt, group)
    assert np.array_equal(np.isnan(onum.to_f32(s, dt)), bad)
    got_c, got_s = codes.cpu().numpy(), onum.to_f32(gen.as_numpy_bits(scales.cpu()), dt)
    assert np.array_equal(got_c, packed) and np.array_equal(got_s, onum.to_f32(s, dt), equal_nan=True)
    keep = np.repeat(~bad, group // 2, axis=1)
    assert np.array_equal(got_c[keep], clean[keep]) and not got_c[~keep].any()
    y = vq.vq_w4_gemv(torch.ones((2, k), dtype=ws.dtype, device=DEV), codes, scales, torch.float32).cpu().numpy()
    assert np.array_equal(np.isnan(y), np.broadcast_to(bad.any(1), (2, n)))


# (rows, outputs, K, group): together every number of parts of K (1 to 16), of waves, of rows a
# workgroup and of loads of x a thread, K that ends inside a chunk of 512 or a piece of 128, parts of
# unequal length and parts of none.
EXACT = [
    (1, 1, 16416, 32), (1, 2048, 4128, 32), (1, 300, 32, 32), (2, 515, 8256, 64), (1, 4100, 4128, 32), (2, 4100, 2208, 32),
    (3, 100, 16416, 32), (4, 515, 8320, 128), (100, 17, 4128, 32), (6, 40, 96, 32), (11, 2048, 8224, 32), (16, 300, 16416, 32),
    (1, 8209, 1056, 32), (2, 12300, 1088, 64), (4, 8209, 2080, 32), (5, 4100, 4128, 32), (8, 4100, 1184, 32),
    (65, 515, 2112, 64), (5, 12300, 1056, 32), (8, 8209, 1152, 128), (16, 4100, 2080, 32),
    (1, 20001, 1056, 32), (3, 16385, 1152, 128), (7, 16385, 1056, 32), (8, 20001, 608, 32), (9, 8209, 2080, 32),
    (13, 12300, 1216, 64), (12, 25001, 1056, 32), (16, 25001, 640, 128), (64, 4100, 1088, 64),
    (17, 16385, 1056, 32), (31, 20001, 576, 64), (32, 28671, 544, 32), (65, 8209, 1184, 32),
]


def whole_numbers(m, n, k, group, dt, seed=0):
    """x of whole numbers up to 7, any code, scales that are powers of two: every partial sum is a
    multiple of 1/4 below 7 * 8 * 2 * K < 2^22, so that float32 holds it exactly in any order."""
    assert 7 * 8 * 2 * k < 2 ** 22
    rng = np.random.default_rng([m, n, k, seed])
    x = gen.to_storage(rng.integers(-7, 8, (m, k)).astype(np.float32), dt)
    packed = rng.integers(0, 256, (n, k // 2), dtype=np.uint8)
    s = gen.to_storage(np.exp2(rng.integers(-2, 2, (n, k // group))).astype(np.float32), dt)
    w = group4.unpack(packed).astype(np.float32) * np.repeat(onum.to_f32(gen.as_numpy_bits(s), dt), group, axis=1)
    return x, packed, s, onum.to_f32(gen.as_numpy_bits(x), dt).astype(np.float64) @ w.astype(np.float64).T


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("m,n,k,group", EXACT)
def test_products_of_whole_numbers_are_exact(vq, m, n, k, group, dt):
    x, packed, s, want = whole_numbers(m, n, k, group, dt)
    y = vq.vq_w4_gemv(x.to(DEV), torch.from_numpy(packed).to(DEV), s.to(DEV), torch.float32)
    assert np.array_equal(y.cpu().numpy().astype(np.float64), want)


@pytest.mark.parametrize("out", ["bf16", "fp16"])
@pytest.mark.parametrize("m,n,k,group", [(1, 4100, 4128, 32), (7, 100, 1056, 32), (20, 515, 640, 128)])
def test_exact_products_are_rounded_once(vq, m, n, k, group, out):
    x, packed, s, want = whole_numbers(m, n, k, group, "bf16")
    y = vq.vq_w4_gemv(x.to(DEV), torch.from_numpy(packed).to(DEV), s.to(DEV), torch.bfloat16 if out == "bf16" else torch.float16)
    with np.errstate(over="ignore"):
        w = onum.from_f32(want.astype(np.float32), out)
    assert np.array_equal(gen.as_numpy_bits(y.cpu()).view(np.uint16) & 0x7FFF, w.view(np.uint16) & 0x7FFF)
    assert np.array_equal(np.sign(onum.to_f32(gen.as_numpy_bits(y.cpu()), out)), np.sign(want))
