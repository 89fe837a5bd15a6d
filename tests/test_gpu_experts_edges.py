"""Experts' products where an index has no row: zeros, whatever the scales and weights hold."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"
TD = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def vq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_quantized_linear_vq_amd as m
    return m


def bad_rows(t):
    rows = torch.arange(t, dtype=torch.int32, device=DEV)
    bad = torch.tensor([0, 3, t // 2, t - 1], device=DEV)
    rows[bad] = torch.tensor([-1, t, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device=DEV)
    keep = torch.ones(t, dtype=torch.bool, device=DEV)
    keep[bad] = False
    return rows, bad, keep


@pytest.mark.parametrize("t", [20, 900])  # either kernel
@pytest.mark.parametrize("out", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("bits", [8, 4])
def test_codes_with_column_scales_that_are_not_finite(vq, t, out, bits):
    e, n, k = 2, 300, 128
    g = torch.Generator(device=DEV).manual_seed(t)
    a = torch.randint(-127, 128, (t, k), device=DEV, generator=g, dtype=torch.int32).to(torch.int8)
    b = torch.randint(0, 256, (e * n, k if bits == 8 else k // 2), device=DEV, generator=g, dtype=torch.int32).to(torch.uint8)
    b = b.view(torch.int8) if bits == 8 else b
    sa, sb = torch.rand(t, device=DEV, generator=g), torch.rand(e * n, device=DEV, generator=g)
    off = torch.tensor([0, t // 3, t], dtype=torch.int32, device=DEV)
    want = vq.vq_qgemm_experts(a, sa, b, sb, bits, off, out_dtype=TD[out])
    rows, bad, keep = bad_rows(t)
    sb2 = sb.clone()
    at = torch.tensor([5, 299], device=DEV)
    for i in range(e):
        sb2[i * n + 5], sb2[i * n + 299] = float("nan"), float("inf")
    y = vq.vq_qgemm_experts(a, sa, b, sb2, bits, off, rows=rows, out_dtype=TD[out])
    assert bool((y[bad] == 0).all())
    cols = torch.ones(n, dtype=torch.bool, device=DEV)
    cols[at] = False
    assert torch.equal(y[keep][:, cols], want[keep][:, cols])
    assert bool(torch.isnan(y[keep][:, 5]).all()) and not bool(torch.isfinite(y[keep][:, 299]).any())


@pytest.mark.parametrize("t", [20, 900])
@pytest.mark.parametrize("out", ["bf16", "fp32"])
def test_rows_and_weights_that_are_not_finite(vq, t, out):
    e, n, k = 2, 300, 128
    g = torch.Generator(device=DEV).manual_seed(t)
    x = torch.randn(t, k, device=DEV, generator=g).bfloat16()
    w = torch.randn(e, n, k, device=DEV, generator=g).bfloat16()
    off = torch.tensor([0, t // 3, t], dtype=torch.int32, device=DEV)
    want = vq.vq_gemm_dense_experts(x, w, off, out_dtype=TD[out])
    rows, bad, keep = bad_rows(t)
    x[0] = float("nan")  # the row that an index without one reads
    w[:, 7, 3] = float("inf")
    y = vq.vq_gemm_dense_experts(x, w, off, rows=rows, out_dtype=TD[out])
    assert bool((y[bad] == 0).all())
    cols = torch.ones(n, dtype=torch.bool, device=DEV)
    cols[7] = False
    assert torch.equal(y[keep][:, cols], want[keep][:, cols]) and not bool(torch.isfinite(y[keep][:, 7]).any())
    assert np.isfinite(want.float().cpu().numpy()).all()
