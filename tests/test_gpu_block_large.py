"""The operators between the layers of a block on tensors of more than 2^31 elements: the last
rows equal those of a small call on the same rows."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def vq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    if torch.cuda.get_device_properties(0).total_memory < 64 << 30:
        pytest.skip("needs 64 GB")
    import bit_quantized_linear_vq_amd as m
    yield m
    torch.cuda.empty_cache()


def half(*shape, seed=0):
    t = torch.empty(*shape, dtype=torch.bfloat16, device=DEV)
    return t.normal_(generator=torch.Generator(device=DEV).manual_seed(seed))


def test_gated_norm(vq):
    m, k = 268500, 8000
    y, h = half(m, k), half(m, k, seed=1)
    mod = torch.randn(m // 4, k // 8, device=DEV).repeat(1, 8)
    n, s = vq.vq_gated_norm(y, h, norm="layer", post="rms", gate=mod, mod_shift=mod)
    at = slice(m - 8, m)
    part = mod[m // 4 - 2:].contiguous()
    n2, s2 = vq.vq_gated_norm(y[at], h[at], norm="layer", post="rms", gate=part, mod_shift=part)
    assert torch.equal(n[at], n2) and torch.equal(s[at], s2)
    del n, s
    codes, scales, s = vq.vq_gated_norm_quant(y, h, 8, norm="layer", post="rms", gate=mod, mod_shift=mod)
    c3, sc3, s3 = vq.vq_gated_norm_quant(y[at], h[at], 8, norm="layer", post="rms", gate=part, mod_shift=part)
    assert torch.equal(codes[at], c3) and torch.equal(scales[at], sc3) and torch.equal(s[at], s3)


def test_combining(vq):
    m, top, n = 140000, 2, 8192
    y = half(m * top, n)
    place = torch.arange(m * top - 1, -1, -1, dtype=torch.int32, device=DEV).view(m, top)
    w = torch.rand(m, top, device=DEV)
    out = vq.vq_combine_experts(y, place, w, out_dtype=torch.float32)
    for at in (slice(0, 5), slice(m - 5, m)):
        rows = place[at].flatten().long()
        want = vq.vq_combine_experts(y[rows].contiguous(), torch.arange(10, dtype=torch.int32, device=DEV).view(5, 2), w[at].contiguous(),
                                     out_dtype=torch.float32)
        assert torch.equal(out[at], want)


@pytest.mark.parametrize("m,n", [(1 << 26, 1), ((1 << 25) + 3, 520)])
def test_combining_of_many_rows(vq, m, n):
    """2^26 pieces of a row and more: 2^32 threads."""
    y = half(16, n)
    place = torch.arange(m, dtype=torch.int32, device=DEV).remainder_(17).view(m, 1)  # the 17th is none
    w = torch.ones(m, 1, device=DEV)
    out = vq.vq_combine_experts(y, place, w)
    want = torch.cat([y, torch.zeros_like(y[:1])])
    whole = m // 17 * 17
    for at in range(0, whole, 17 << 18):
        part = out[at:min(whole, at + (17 << 18))].view(-1, 17, n)
        assert bool((part == want).all()), at
    assert torch.equal(out[whole:], want[:m - whole])


@pytest.mark.parametrize("m,n,k", [(80000, 28672, 64), (270000, 16, 8192)])
def test_adapters(vq, m, n, k):
    x, base = half(m, k), half(m, n, seed=1)
    down, up = half(2, 8, k, seed=2) * 0.1, half(2, n, 8, seed=3)
    index = torch.randint(-1, 2, (m,), device=DEV, dtype=torch.int32)
    out = vq.vq_lowrank_add(base, x, down, up, index)
    for at in (slice(0, 40), slice(m - 40, m)):
        # the parts of K may differ: equal but for the rounding of sums in another order
        want = vq.vq_lowrank_add(base[at], x[at], down, up, index[at].contiguous())
        assert torch.allclose(out[at].float(), want.float(), rtol=2.0 ** -7, atol=1e-4)


def test_many_large_adapters(vq):
    """Adapters' offsets beyond 2^31 elements."""
    ad, k, n, r = 2100, 8192, 8192, 128
    down, up = half(ad, r, k) * (k ** -0.5), half(ad, n, r, seed=1)
    index = torch.tensor([0, ad - 1, ad, 7, ad - 1], dtype=torch.int32, device=DEV)
    x, base = half(5, k, seed=2), half(5, n, seed=3)
    out = vq.vq_lowrank_add(base, x, down, up, index)
    small = vq.vq_lowrank_add(base, x, down[[0, 7, ad - 1]].contiguous(), up[[0, 7, ad - 1]].contiguous(),
                              torch.tensor([0, 2, -1, 1, 2], dtype=torch.int32, device=DEV))
    assert torch.equal(out, small)


def test_routing_of_many_rows(vq):
    m, e, top = 1 << 21, 64, 8
    x = torch.randn(m, e, device=DEV)
    off, rows, w, ch, place = vq.vq_route_experts(x, top)
    torch.cuda.synchronize()
    # (topk leaves the order of equal scores open)
    assert torch.equal(ch.long(), torch.sort(x, dim=1, descending=True, stable=True).indices[:, :top])
    assert int(off[e]) == m * top and torch.equal(rows[place.flatten().long()], torch.arange(m, device=DEV, dtype=torch.int32).repeat_interleave(top))
    sorted_ch = torch.empty(m * top, dtype=torch.int32, device=DEV)
    sorted_ch[place.flatten().long()] = ch.flatten()
    assert bool((sorted_ch[1:] >= sorted_ch[:-1]).all())
    same = sorted_ch[1:] == sorted_ch[:-1]
    assert bool((rows[1:] >= rows[:-1])[same].all())
