"""The norm to codes in the layouts of long calls: rows of one, two or more waves, several rows to a
workgroup, more rows than one pass of the grid, each with and without the outlier partition
and with the width and the scales from the device.  Bit for bit, as the formula gives it."""
import numpy as np
import pytest
import torch

import gen
from oracle import norm as onorm

pytestmark = pytest.mark.gpu

DEV = "cuda"
EPS = 1e-6


@pytest.fixture(scope="module")
def vq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_quantized_linear_vq_amd as m
    return m


def make(m, k, dt, res, seed=0):
    rng = np.random.default_rng([m, k, seed])
    x = rng.standard_normal((m, k)).astype(np.float32)
    x[:, :: max(1, k // 19)] *= 20.0
    r = gen.to_storage((2 * rng.standard_normal((m, k))).astype(np.float32), dt) if res else None
    return gen.to_storage(x, dt), r, (1 + 0.2 * rng.standard_normal(k)).astype(np.float32)


def outliers(k, n):
    return np.sort(np.random.default_rng([k, n]).choice(k, n, replace=False)).astype(np.int32) if n else None


def bits(t):
    return np.ascontiguousarray(gen.as_numpy_bits(t.cpu())).view(np.uint16)


@pytest.mark.parametrize("m,k,n_out,dt,res", [
    (1500, 1920, 19, "bf16", True), (1500, 1920, 128, "fp16", False), (1025, 2048, 1, "bf16", True),  # a wave a row, four rows
    (50, 640, 70, "bf16", True), (51, 1024, 9, "fp16", True), (1023, 576, 65, "bf16", False),  # two waves, one piece a thread
    (1100, 4096, 64, "bf16", True), (1029, 2112, 3, "fp16", True),  # two waves, four pieces
    (1040, 5760, 100, "bf16", True), (1031, 12288, 17, "bf16", False), (1027, 32768, 128, "bf16", True),  # three to sixteen
])
@pytest.mark.parametrize("gran", ["token", "static"])
def test_outlier_partition_in_every_layout(vq, m, k, n_out, dt, res, gran):
    x, r, w = make(m, k, dt, res)
    idx = outliers(k, n_out)
    st = np.array([0.03, 0.4], np.float32) if gran == "static" else None
    got = vq.vq_rmsnorm_quant(x.to(DEV), torch.from_numpy(w).to(DEV), 8, EPS, residual=r.to(DEV) if res else None, gran=gran,
                              idx=torch.from_numpy(idx).to(DEV), static_scale=None if st is None else torch.from_numpy(st).to(DEV))
    torch.cuda.synchronize()
    h, v = onorm.rows(gen.as_numpy_bits(x), dt, w, EPS, gen.as_numpy_bits(r) if res else None)
    codes, scales = onorm.quant(v, 8, idx, st)
    assert np.array_equal(got[1].cpu().numpy().reshape(-1).view(np.uint32), scales.reshape(-1).view(np.uint32))
    assert np.array_equal(got[0].cpu().numpy(), codes)
    if res:
        assert np.array_equal(bits(got[2]), np.ascontiguousarray(h).view(np.uint16))


@pytest.mark.parametrize("m,k", [(9000, 4096), (5000, 12288), (4500, 5760), (20000, 640)])
@pytest.mark.parametrize("n_out", [0, 40])
def test_more_rows_than_a_pass_of_the_grid(vq, m, k, n_out):
    """The whole call, the sum in place, against calls of few rows (which the oracle pins)."""
    g = torch.Generator(device=DEV).manual_seed(m + k)
    x = torch.randn(m, k, device=DEV, generator=g).bfloat16()
    r = torch.randn(m, k, device=DEV, generator=g).bfloat16()
    x[:: 7] *= 5.0
    w = torch.randn(k, device=DEV, generator=g).bfloat16()
    idx = torch.from_numpy(outliers(k, n_out)).to(DEV) if n_out else None
    nb = torch.tensor([6], dtype=torch.int32, device=DEV)
    for kw in (dict(), dict(bits_dev=nb), dict(gran="static", static_scale=torch.tensor([0.02, 0.3], device=DEV)[:2 if n_out else 1])):
        h = r.clone()
        codes, scales = vq.vq_rmsnorm_quant(x, w, 8, EPS, residual=h, sum_out=h, idx=idx, **kw)[:2]
        for i in range(0, m, 950):
            s = slice(i, min(m, i + 950))
            c, sc, hs = vq.vq_rmsnorm_quant(x[s], w, 8, EPS, residual=r[s], idx=idx, **kw)
            assert torch.equal(codes[s], c) and torch.equal(h[s], hs)
            assert torch.equal(scales[s] if "gran" not in kw else scales, sc)


def test_few_rows_that_the_long_calls_are_held_to(vq):
    """The oracle's pin of the calls that the test above compares with, widths and scales too."""
    for k, n_out in ((4096, 40), (12288, 40), (5760, 40), (640, 40), (4096, 0), (12288, 0)):
        x, r, w = make(30, k, "bf16", True, 3)
        idx = outliers(k, n_out)
        st = np.array([0.02, 0.3], np.float32)[:2 if n_out else 1]
        for nb, kw in ((8, dict()), (6, dict(bits_dev=torch.tensor([6], dtype=torch.int32, device=DEV))),
                       (8, dict(gran="static", static_scale=torch.from_numpy(st).to(DEV)))):
            c, s, h = vq.vq_rmsnorm_quant(x.to(DEV), torch.from_numpy(w).to(DEV), 8, EPS, residual=r.to(DEV),
                                          idx=None if idx is None else torch.from_numpy(idx).to(DEV), **kw)
            oh, v = onorm.rows(gen.as_numpy_bits(x), "bf16", w, EPS, gen.as_numpy_bits(r))
            codes, scales = onorm.quant(v, nb, idx, st if "gran" in kw else None)
            assert np.array_equal(c.cpu().numpy(), codes) and np.array_equal(bits(h), np.ascontiguousarray(oh).view(np.uint16))
            assert np.array_equal(s.cpu().numpy().reshape(-1).view(np.uint32), scales.reshape(-1).view(np.uint32))
