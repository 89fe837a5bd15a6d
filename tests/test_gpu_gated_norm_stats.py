"""Statistics of the layer norm in rows that hardly differ from a large mean, bit for bit (oracle/gated.py).

S2 / K - mean^2 in float64 is off by 2^-53 (mean / deviation)^2 of itself: tens of float32 steps here.  The sums
S1 and S2 of such rows are exact in float64, so (K S2 - S1^2) / K^2 without rounded products is too, but for 2^-52 of it.
"""
import numpy as np
import pytest
import torch

import gen
from oracle import gated as og
from oracle import norm as onorm
from oracle import numerics as onum

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def vq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_quantized_linear_vq_amd as m
    return m


def nearly_constant(m, k, big, step, some, seed=0):
    """Rows of `big`, of whose elements up to `some` are one or two steps higher, the first one in every other row."""
    rng = np.random.default_rng([m, k, int(abs(big)), seed])
    x = np.full((m, k), big, np.float32)
    for i in range(m):
        n = int(rng.integers(1, min(some, k) + 1))
        at = rng.choice(k, n, replace=False)
        x[i, at] += step * rng.integers(1, 3, n).astype(np.float32)
        if i % 2:
            x[i, 0] = big + step
    return gen.to_storage(x, "fp16")


def words(t):
    a = gen.as_numpy_bits(t.cpu().contiguous()) if isinstance(t, torch.Tensor) else np.ascontiguousarray(t)
    return a.view(np.uint16 if a.dtype.itemsize == 2 else np.uint32 if a.dtype.itemsize == 4 else a.dtype)


@pytest.mark.parametrize("m,k,big,step,some", [(400, 12288, 2000.0, 1.0, 5), (400, 1920, 100.0, 0.0625, 6), (1100, 4096, 4000.0, 2.0, 9),
                                               (1030, 1920, 60000.0, 32.0, 3), (1025, 16384, 1000.0, 0.5, 40), (9, 64, 2000.0, 1.0, 2)])
def test_codes_and_scales_of_nearly_constant_rows(vq, m, k, big, step, some):
    h = nearly_constant(m, k, big, step, some)
    codes, scales, _ = vq.vq_gated_norm_quant(None, h.to(DEV), 8, norm="layer")
    torch.cuda.synchronize()
    _, v = og.rows(None, gen.as_numpy_bits(h), "fp16", "layer")
    oc, osc = onorm.quant(v, 8)
    assert np.array_equal(words(scales), words(osc).reshape(-1))
    assert np.array_equal(codes.cpu().numpy(), oc)


@pytest.mark.parametrize("m,k,big,step", [(600, 12288, 2000.0, 1.0), (600, 4099, 2000.0, 1.0), (1100, 2055, 500.0, 0.25), (40, 7, 2000.0, 1.0),
                                          (1024, 16390, 1000.0, 0.5)])
def test_rows_and_branches_that_are_nearly_constant(vq, m, k, big, step):
    """Both norms, in rows of every kind of end."""
    h, y = nearly_constant(m, k, big, step, 4), nearly_constant(m, k, -big, step, 4, seed=1)
    g = np.full((1, k), 1.0, np.float32)
    w = np.linspace(0.5, 1.5, k).astype(np.float32)
    n, s = vq.vq_gated_norm(y.to(DEV), h.to(DEV), torch.from_numpy(w).to(DEV), norm="layer", post="layer", post_weight=torch.from_numpy(w).to(DEV),
                            gate=torch.from_numpy(g).to(DEV))
    torch.cuda.synchronize()
    os_, ov = og.rows(gen.as_numpy_bits(y), gen.as_numpy_bits(h), "fp16", "layer", w, 1e-6, "layer", w, 1.0, g)
    assert np.array_equal(words(s), words(os_)) and np.array_equal(words(n), words(onum.from_f32(ov, "fp16")))


@pytest.mark.parametrize("k", [1, 8, 64, 1920, 4099, 8192])
@pytest.mark.parametrize("value", [60000.0, -3.0, 1e-7])
def test_constant_rows_are_zero_with_any_eps(vq, k, value):
    h = torch.full((3, k), value, dtype=torch.float16, device=DEV)
    for eps in (1e-6, 1e-30):
        n, _ = vq.vq_gated_norm(None, h, norm="layer", eps=eps)
        assert not n.any()


@pytest.mark.parametrize("m", [3, 1100])
@pytest.mark.parametrize("k", [512, 4096, 8192])
@pytest.mark.parametrize("norm", ["rms", "layer"])
def test_an_infinity_or_nan_anywhere_in_a_row(vq, norm, k, m):
    """In the first element, another wave's, or the last."""
    h = torch.randn(m, k, device=DEV, generator=torch.Generator(device=DEV).manual_seed(k)).half()
    good, _ = vq.vq_gated_norm(None, h, norm=norm)
    for at in (0, 1, k // 2, k - 1):
        for v in (float("inf"), float("-inf"), float("nan")):
            x = h.clone()
            x[1, at] = v
            n, _ = vq.vq_gated_norm(None, x, norm=norm)
            want = torch.zeros(k, device=DEV)
            want[at] = float("nan")  # rms of an infinity: 1 / inf of the others, inf * 0 there
            if norm == "layer" or v != v:
                want[:] = float("nan")
            assert torch.equal(n[1].float().nan_to_num(7.0), want.nan_to_num(7.0)), (at, v)
            assert torch.equal(n[[0, 2]], good[[0, 2]])


def test_rows_outside_the_sets_keep_every_bit(vq):
    """Also those of a NaN, quiet or signaling, and of numbers below the normal range."""
    for dt, odd in ((torch.bfloat16, [0x7F81, 0x7FC1, 0xFFFF, 0x7F80, 0x0001, 0x8000]), (torch.float16, [0x7C01, 0x7E55, 0xFFFF, 0x7C00, 0x0001, 0x8000])):
        h = torch.randn(6, 256, device=DEV).to(dt)
        h.view(torch.int16)[3, 10:16] = torch.tensor(odd, dtype=torch.int32).to(torch.int16).to(DEV)
        index = torch.tensor([0, 1, 0, 2, 1, -1], dtype=torch.int32, device=DEV)
        for post in (None, "rms"):
            _, s = vq.vq_gated_norm(torch.randn_like(h), h, post=post, gate=torch.ones(2, 256, device=DEV), index=index)
            assert torch.equal(s.view(torch.int16)[[3, 5]], h.view(torch.int16)[[3, 5]])
