"""A prepared function's own tensors stay its own: what the allocator hands out afterwards is not
written to, and the results follow the inputs."""
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


def test_tensors_that_a_prepared_function_drops(vq):
    g = torch.Generator(device=DEV).manual_seed(1)
    x, r = (torch.randn(48, 256, device=DEV, generator=g).bfloat16() for _ in range(2))
    w = (torch.randn(2 * 96, 256, device=DEV, generator=g) * 0.05).bfloat16()
    down = (torch.randn(2 * 256, 96 // 32 * 64, device=DEV, generator=g) * 0.05).bfloat16()
    wc, ws = vq.vq_pack_weights(w, 8)
    off = torch.tensor([0, 20, 48], dtype=torch.int32, device=DEV)

    def f(x, r):
        c, s, h = vq.vq_rmsnorm_quant(x, None, 8, residual=r)
        mid = vq.vq_qgemm_experts(c, s, wc, ws, 8, off)
        wide = torch.empty(48, 192, dtype=torch.bfloat16, device=DEV)
        vq.vq_gemm_dense(mid[:, :64], down[:192, :64].contiguous(), y=wide)
        return vq.vq_gemm_dense_experts(wide, down.view(2, 256, 192), off)

    launch, y = vq.prepare(f, x, r)
    torch.cuda.synchronize()
    others = [torch.full((n,), 7, dtype=torch.uint8, device=DEV) for n in (48 * 256, 192, 48 * 512, 48 * 192, 48 * 384, 192 * 128) for _ in range(40)]
    for _ in range(3):
        x.copy_(torch.randn(48, 256, device=DEV, generator=g))
        y.zero_()
        launch()
        want = f(x, r)
        torch.cuda.synchronize()
        assert torch.equal(y, want)
    assert all(bool((t == 7).all()) for t in others)
