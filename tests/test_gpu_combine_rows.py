"""Combining: rows whose index is outside the gate's sets."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def vq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_quantized_linear_vq_amd as m
    return m


@pytest.mark.parametrize("n", [5, 256, 1003])
@pytest.mark.parametrize("dt,odd", [(torch.bfloat16, [0x7F81, 0xFFFF, 0x7F80, 0x0001, 0x8000]), (torch.float16, [0x7C01, 0xFFFF, 0x7C00, 0x0001, 0x8000])])
def test_rows_outside_the_sets_keep_every_bit(vq, dt, odd, n):
    """Also those of a signaling NaN; the other rows are gated, in place or not."""
    res = torch.randn(6, n, device=DEV).to(dt)
    res.view(torch.int16)[3, :5] = torch.tensor(odd, dtype=torch.int32).to(torch.int16).to(DEV)
    index = torch.tensor([0, 1, 0, 2, 1, -1], dtype=torch.int32, device=DEV)
    y, w = torch.randn(12, n, device=DEV).to(dt), torch.rand(6, 2, device=DEV)
    place = torch.arange(12, dtype=torch.int32, device=DEV).view(6, 2)
    gate = torch.rand(2, n, device=DEV)
    out = vq.vq_combine_experts(y, place, w, residual=res, gate=gate, index=index)
    assert torch.equal(out.view(torch.int16)[[3, 5]], res.view(torch.int16)[[3, 5]])
    each = vq.vq_combine_experts(y, place, w, residual=res, gate=gate[index.long().clamp(0, 1)].contiguous())
    assert torch.equal(out[[0, 1, 2, 4]], each[[0, 1, 2, 4]])
    same = res.clone()
    vq.vq_combine_experts(y, place, w, residual=same, gate=gate, index=index, out=same)
    assert torch.equal(same.view(torch.int16), out.view(torch.int16))
