"""GPU parity of group-scaled 4-bit weights: the packing bit for bit, the product with a few
rows within the bound of its float32 sums (oracle/group4.py) plus half a step of the output
type."""
import numpy as np
import pytest
import torch

import gen
from oracle import group4
from oracle import numerics as onum

pytestmark = pytest.mark.gpu

DEV = "cuda"
TD = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def vq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_quantized_linear_vq_amd as m
    return m


def npb(t):
    t = t.cpu().contiguous()
    return t.numpy() if t.dtype == torch.float32 else gen.as_numpy_bits(t)


def within(y, ex, b, out):
    got = y.float().cpu().numpy().astype(np.float64)
    if out != "fp32":
        mant, emin = (7, -126) if out == "bf16" else (10, -14)
        b = b + 0.5 * np.exp2(np.floor(np.log2(np.maximum(np.abs(ex) + b, 2.0 ** emin))) - mant)
    err = np.abs(got - ex)
    assert np.all(err <= b + 1e-300), float((err / np.maximum(b, 1e-300)).max())


@pytest.mark.parametrize("n,k,group,dt", [
    (1, 32, 32, "bf16"), (3, 64, 64, "fp16"), (5, 128, 128, "bf16"), (37, 1920, 128, "bf16"),
    (300, 480, 32, "fp16"), (7, 12288, 64, "bf16"), (129, 96, 32, "bf16"),
])
def test_packing(vq, n, k, group, dt):
    rng = np.random.default_rng([n, k, group])
    w = (rng.standard_normal((n, k)) * 0.02).astype(np.float32)
    w[0, : min(group, k)] = 0.0  # a group of zeros
    w[-1, -group:] *= 1e-3 if dt == "fp16" else 1e-30
    ws = gen.to_storage(w, dt)
    codes, scales = vq.vq_pack_weights_group(ws.to(DEV), group)
    torch.cuda.synchronize()
    _, packed, s = group4.pack(gen.as_numpy_bits(ws), dt, group)
    assert np.array_equal(npb(scales).view(np.uint16), np.asarray(s).view(np.uint16))
    assert np.array_equal(codes.cpu().numpy(), packed)


CASES = [
    (1, 1, 32, 32, "bf16", "bf16"), (1, 5, 64, 64, "fp16", "fp32"), (1, 1920, 1920, 128, "bf16", "bf16"),
    (2, 33, 96, 32, "fp16", "fp16"), (3, 255, 4096, 64, "bf16", "fp32"), (7, 1000, 480, 32, "fp16", "fp16"),
    (8, 64, 12288, 128, "bf16", "fp16"), (16, 130, 640, 128, "fp16", "bf16"), (17, 96, 1024, 64, "bf16", "bf16"),
    (31, 40, 160, 32, "bf16", "fp32"), (33, 70, 384, 128, "fp16", "fp16"), (64, 17, 256, 32, "bf16", "bf16"),
    (100, 48, 8192, 128, "fp16", "fp32"), (1, 4097, 128, 128, "bf16", "fp32"), (5, 16, 16416, 32, "bf16", "fp32"),
]


@pytest.mark.parametrize("m,n,k,group,dt,out", CASES)
def test_product_within_the_float32_bound(vq, m, n, k, group, dt, out):
    rng = np.random.default_rng([m, n, k])
    x = gen.to_storage((rng.standard_normal((m, k)) + 0.5).astype(np.float32), dt)
    w = gen.to_storage((rng.standard_normal((n, k)) * 0.02).astype(np.float32), dt)
    codes, scales = vq.vq_pack_weights_group(w.to(DEV), group)
    y = vq.vq_w4_gemv(x.to(DEV), codes, scales, TD[out])
    torch.cuda.synchronize()
    ex, b = group4.exact(gen.as_numpy_bits(x), dt, codes.cpu().numpy(), npb(scales), group)
    within(y, ex, b, out)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("m,group", [(1, 32), (4, 64), (20, 128)])
def test_every_nibble_at_every_place(vq, m, group, dt):
    """All sixteen nibbles (-8 too) at every position of a group, against unit rows: each
    output is one code times its scale, exact in float32."""
    k = group
    n = 16
    c = np.empty((n, k), dtype=np.int64)
    for j in range(n):
        c[j] = (np.arange(k) * 5 + j) % 16
    packed = (c[:, 0::2] | (c[:, 1::2] << 4)).astype(np.uint8)
    s = gen.to_storage(np.full((n, 1), 0.5, dtype=np.float32), dt)
    want = np.where(c > 7, c - 16, c) * 0.5
    for at in range(0, k, m):
        rows = min(m, k - at)
        x = np.zeros((rows, k), dtype=np.float32)
        x[np.arange(rows), at + np.arange(rows)] = 1.0
        y = vq.vq_w4_gemv(gen.to_storage(x, dt).to(DEV), torch.from_numpy(packed).to(DEV), s.to(DEV), torch.float32)
        assert np.array_equal(y.cpu().numpy(), want.T[at:at + rows].astype(np.float32))


def test_rows_do_not_depend_on_their_neighbours(vq):
    """An infinity or NaN stays in its row."""
    rng = np.random.default_rng(5)
    x = gen.to_storage(rng.standard_normal((9, 1920)).astype(np.float32), "bf16").to(DEV)
    w = gen.to_storage((rng.standard_normal((100, 1920)) * 0.02).astype(np.float32), "bf16").to(DEV)
    codes, scales = vq.vq_pack_weights_group(w, 64)
    y = vq.vq_w4_gemv(x, codes, scales, torch.float32)
    x2 = x.clone()
    x2[3, 7] = float("nan")
    x2[5, 1919] = float("inf")
    y2 = vq.vq_w4_gemv(x2, codes, scales, torch.float32)
    keep = torch.tensor([0, 1, 2, 4, 6, 7, 8], device=DEV)
    assert torch.equal(y2[keep], y[keep])
    assert bool(torch.isnan(y2[3]).all()) and not bool(torch.isfinite(y2[5]).any())


def test_pitches(vq):
    rng = np.random.default_rng(6)
    m, n, k = 5, 77, 256
    xf = gen.to_storage(rng.standard_normal((m, k + 40)).astype(np.float32), "fp16").to(DEV)
    w = gen.to_storage((rng.standard_normal((n, k + 64)) * 0.02).astype(np.float32), "fp16").to(DEV)
    codes, scales = vq.vq_pack_weights_group(w[:, :k], 32)
    c2, s2 = vq.vq_pack_weights_group(w[:, :k].contiguous(), 32)
    assert torch.equal(codes, c2) and torch.equal(scales, s2)
    big = torch.full((m, n + 3), 7.0, dtype=torch.float16, device=DEV)
    vq.vq_w4_gemv(xf[:, :k], codes, scales, y=big[:, :n])
    want = vq.vq_w4_gemv(xf[:, :k].contiguous(), codes, scales)
    assert torch.equal(big[:, :n], want) and bool((big[:, n:] == 7.0).all())


def test_no_rows_and_refusals(vq):
    w = torch.randn(16, 128, device=DEV).to(torch.bfloat16)
    codes, scales = vq.vq_pack_weights_group(w, 64)
    x = torch.zeros((2, 128), dtype=torch.bfloat16, device=DEV)
    assert vq.vq_w4_gemv(x[:0], codes, scales).shape == (0, 16)
    with pytest.raises(ValueError):
        vq.vq_pack_weights_group(w, 48)
    with pytest.raises(ValueError):
        vq.vq_pack_weights_group(w[:, :96], 64)
    with pytest.raises(TypeError):
        vq.vq_pack_weights_group(w.float(), 64)
    with pytest.raises(TypeError):
        vq.vq_w4_gemv(x.half(), codes, scales)
    with pytest.raises(ValueError):
        vq.vq_w4_gemv(x[:, :64], codes, scales)
    with pytest.raises(ValueError):
        vq.vq_w4_gemv(x, codes, scales[:8].contiguous())
    with pytest.raises(vq.VQError):
        vq.vq_w4_gemv(x, codes, torch.ones((16, 8), dtype=torch.bfloat16, device=DEV))  # groups of 16
    with pytest.raises(ValueError):
        vq.vq_w4_gemv(x, codes, scales, y=torch.empty((2, 15), dtype=torch.bfloat16, device=DEV))


def test_captured_and_replayed(vq):
    rng = np.random.default_rng(8)
    w = gen.to_storage((rng.standard_normal((1920, 1920)) * 0.02).astype(np.float32), "bf16").to(DEV)
    codes, scales = vq.vq_pack_weights_group(w, 128)
    xs = [gen.to_storage(rng.standard_normal((2, 1920)).astype(np.float32), "bf16").to(DEV) for _ in range(3)]
    x = xs[0].clone()
    y = torch.empty((2, 1920), dtype=torch.bfloat16, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            vq.vq_w4_gemv(x, codes, scales, y=y)
    torch.cuda.synchronize()
    for t in xs + xs[:1]:
        x.copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, vq.vq_w4_gemv(t, codes, scales))


@pytest.mark.parametrize("m,n,k,group", [(1, 20000, 128, 64), (2, 30, 4128, 32), (9, 33, 640, 64), (16, 2048, 4096, 128)])
def test_products_of_small_values(vq, m, n, k, group):
    """fp16 rows and scales below the normal range: nothing is flushed to zero."""
    rng = np.random.default_rng([m, n])
    x = gen.to_storage((rng.standard_normal((m, k)) * 2e-6).astype(np.float32), "fp16")
    w = gen.to_storage((rng.standard_normal((n, k)) * 2e-4).astype(np.float32), "fp16")
    codes, scales = vq.vq_pack_weights_group(w.to(DEV), group)
    y = vq.vq_w4_gemv(x.to(DEV), codes, scales, torch.float32)
    torch.cuda.synchronize()
    _, packed, s = group4.pack(gen.as_numpy_bits(w), "fp16", group)
    assert np.array_equal(codes.cpu().numpy(), packed)
    assert np.array_equal(npb(scales).view(np.uint16), np.asarray(s).view(np.uint16))
    ex, b = group4.exact(gen.as_numpy_bits(x), "fp16", packed, s, group)
    within(y, ex, b, "fp32")


@pytest.mark.parametrize("m,n,k,group,dt,out", [
    (16, 16500, 1056, 32, "bf16", "bf16"), (12, 25001, 640, 128, "fp16", "fp32"), (9, 24600, 320, 64, "bf16", "fp16"),
    (16, 16385, 32, 32, "fp16", "bf16"), (8, 8209, 1056, 32, "bf16", "fp32"), (7, 12300, 1280, 128, "fp16", "fp16"),
    (5, 12500, 2112, 64, "bf16", "bf16"), (8, 8192, 640, 128, "bf16", "bf16"),
])
def test_many_channels_with_many_rows(vq, m, n, k, group, dt, out):
    test_product_within_the_float32_bound(vq, m, n, k, group, dt, out)


@pytest.mark.parametrize("m,n,k,group,dt,out", [
    (17, 100, 1056, 32, "bf16", "bf16"), (32, 65, 32, 32, "fp16", "fp32"), (33, 1000, 640, 128, "bf16", "fp16"),
    (24, 17000, 1088, 64, "bf16", "bf16"), (31, 129, 8320, 64, "fp16", "bf16"), (65, 40, 2080, 32, "bf16", "fp32"),
])
def test_more_rows_than_a_tile(vq, m, n, k, group, dt, out):
    test_product_within_the_float32_bound(vq, m, n, k, group, dt, out)


@pytest.mark.parametrize("m,n,k,group,dt,out", [
    (5, 50, 2080, 32, "bf16", "bf16"), (6, 333, 1088, 64, "fp16", "fp32"), (11, 40, 4224, 128, "bf16", "fp16"),
    (16, 515, 2112, 64, "bf16", "bf16"), (13, 3001, 352, 32, "fp16", "bf16"), (21, 1999, 480, 32, "bf16", "fp32"),
    (32, 4100, 320, 64, "bf16", "bf16"), (67, 30, 8192, 128, "fp16", "fp16"), (130, 100, 96, 32, "bf16", "bf16"),
])
def test_rows_in_smaller_tiles(vq, m, n, k, group, dt, out):
    test_product_within_the_float32_bound(vq, m, n, k, group, dt, out)
