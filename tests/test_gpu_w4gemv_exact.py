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
