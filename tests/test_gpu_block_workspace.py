"""One scratch, made for a program's largest call, for all of its smaller ones: the same results, and nothing
written behind it."""
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


@pytest.mark.parametrize("k,r,adapters", [(8192, 32, 5), (4096, 64, 16), (2048, 128, 3)])
def test_adapters(vq, k, r, adapters):
    most, n = 17776, 24
    g = torch.Generator(device=DEV).manual_seed(k)
    x = torch.empty(most, k, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    base = torch.empty(most, n, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    down = (torch.randn(adapters, r, k, device=DEV, generator=g) * k ** -0.5).bfloat16()
    up = torch.randn(adapters, n, r, device=DEV, generator=g).bfloat16()
    index = torch.randint(-1, adapters, (most,), device=DEV, generator=g, dtype=torch.int32)
    need = vq.vq_lowrank_workspace_elems(most, adapters, r, k)
    ws = torch.full((need + 4096,), 9.0, device=DEV)
    for m in (1, 17, 256, 513, 4000, 8192, 12000, 16000, most):
        for a in {1, adapters}:
            args = (base[:m], x[:m], down[:a], up[:a], index[:m])
            assert torch.equal(vq.vq_lowrank_add(*args, ws=ws[:need]), vq.vq_lowrank_add(*args)), (m, a)
    assert bool((ws[need:] == 9.0).all())


@pytest.mark.parametrize("e", [8, 160, 300, 1024])
def test_routing(vq, e):
    most, top = 100000, 4
    x = torch.randn(most, e, device=DEV, generator=torch.Generator(device=DEV).manual_seed(e))
    need = vq.vq_route_experts_workspace_elems(most, e)
    ws = torch.full((need + 4096,), 77, dtype=torch.int32, device=DEV)
    for m in (1, 65, 684, 1000, 2000, 2049, 17776, 50000, most):
        got = vq.vq_route_experts(x[:m], top, ws=ws[:need])
        assert all(torch.equal(a, b) for a, b in zip(got, vq.vq_route_experts(x[:m], top))), m
    assert bool((ws[need:] == 77).all())
