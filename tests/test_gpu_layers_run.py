"""The norm, the experts' products, the quantizer and the single-token product as a block of a
network runs them.

A feed-forward block over experts: norm with the residual to codes, the gate's rows sorted
by expert, the up product, the quantizer, the down product.  Every step's outputs follow
from exact integers and single roundings, so the block's result must equal the oracle's
chain bit for bit, eagerly and from a graph replayed with other inputs and offsets.  And one
token through the norm and the group-scaled product, against the exact product of the
oracle's normed row within the float32 bound.
"""
import numpy as np
import pytest
import torch

import gen
from oracle import group4, quantizer
from oracle import norm as onorm
from oracle import numerics as onum

pytestmark = pytest.mark.gpu

DEV = "cuda"
EPS = 1e-5


@pytest.fixture(scope="module")
def vq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_quantized_linear_vq_amd as m
    return m


def bits(t):
    return gen.as_numpy_bits(t.cpu().contiguous())


def oracle_product(codes, scales, w_codes, w_scales, off, rows, n):
    y = np.zeros((len(rows), n), np.float32)
    for e in range(len(off) - 1):
        i = rows[off[e]:off[e + 1]]
        b = w_codes[e * n:(e + 1) * n]
        acc = codes[i].astype(np.float64) @ b.astype(np.float64).T
        s = (scales[i][:, None] * w_scales[None, e * n:(e + 1) * n]).astype(np.float32)
        y[off[e]:off[e + 1]] = (acc.astype(np.float32) * s).astype(np.float32)
    return onum.from_f32(y, "bf16")


@pytest.mark.parametrize("tokens,w_bits,kblock", [(3, 8, True), (90, 4, False), (700, 8, True)])
def test_block_over_experts(vq, tokens, w_bits, kblock):
    dim, hidden, e, top = 320, 640, 5, 2
    rng = np.random.default_rng(tokens)

    def half(*shape, scale=1.0):
        return gen.to_storage((rng.standard_normal(shape) * scale).astype(np.float32), "bf16")
    up, down = half(e * hidden, dim, scale=0.05), half(e * dim, hidden, scale=0.05)
    wn = half(dim)
    uc, us = vq.vq_pack_weights(up.to(DEV), w_bits, kblock=kblock)
    dc, ds = vq.vq_pack_weights(down.to(DEV), w_bits, kblock=kblock)
    ou, _, ous = quantizer.pack_weights(gen.as_numpy_bits(up), "bf16", w_bits)
    od, _, ods = quantizer.pack_weights(gen.as_numpy_bits(down), "bf16", w_bits)
    t = tokens * top
    x, r = half(tokens, dim).to(DEV), half(tokens, dim).to(DEV)
    off = torch.zeros(e + 1, dtype=torch.int32, device=DEV)
    rows = torch.zeros(t, dtype=torch.int32, device=DEV)
    out = [torch.empty(tokens, dim, dtype=torch.int8, device=DEV), torch.empty(tokens, device=DEV),
           torch.empty(tokens, dim, dtype=torch.bfloat16, device=DEV),
           torch.empty(t, hidden, dtype=torch.bfloat16, device=DEV),
           torch.empty(t, hidden, dtype=torch.int8, device=DEV), torch.empty(t, device=DEV),
           torch.empty(t, dim, dtype=torch.bfloat16, device=DEV)]
    wnd = wn.to(DEV)

    def step():
        c, s, h, mid, c2, s2, y = out
        vq.vq_rmsnorm_quant(x, wnd, 8, EPS, residual=r, codes=c, scales=s, sum_out=h)
        vq.vq_qgemm_experts(c, s, uc, us, w_bits, off, rows=rows, y=mid)
        vq.vq_quant_act(mid, 8, "token", codes=c2, scales=s2)
        vq.vq_qgemm_experts(c2, s2, dc, ds, w_bits, off, y=y)

    def new_inputs(seed):
        g = np.random.default_rng(seed)
        x.copy_(gen.to_storage(g.standard_normal((tokens, dim)).astype(np.float32), "bf16"))
        r.copy_(gen.to_storage(g.standard_normal((tokens, dim)).astype(np.float32), "bf16"))
        pick = g.integers(0, e, t) if seed % 2 else np.minimum(g.integers(0, 2 * e, t), e - 1)
        order = np.argsort(pick, kind="stable")
        off.copy_(torch.from_numpy(np.concatenate([[0], np.cumsum(np.bincount(pick, minlength=e))]).astype(np.int32)))
        rows.copy_(torch.from_numpy((order // top).astype(np.int32)))

    def check():
        torch.cuda.synchronize()
        o, i = off.cpu().numpy(), rows.cpu().numpy()
        h, v = onorm.rows(bits(x), "bf16", onum.to_f32(gen.as_numpy_bits(wn), "bf16"), EPS, bits(r))
        c, s = onorm.quant(v, 8)
        mid = oracle_product(c, s, ou, ous, o, i, hidden)
        c2, s2 = quantizer.quant_act(mid, "bf16", 8, "token")
        y = oracle_product(c2, s2, od, ods, o, np.arange(t), dim)
        assert np.array_equal(bits(out[2]), h)
        assert np.array_equal(out[0].cpu().numpy(), c) and np.array_equal(out[1].cpu().numpy(), s)
        assert np.array_equal(bits(out[3]), mid)
        assert np.array_equal(bits(out[6]), y)

    new_inputs(1)
    step()
    check()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            step()
    torch.cuda.synchronize()
    for seed in (2, 3, 4):
        new_inputs(seed)
        for o in out:
            o.zero_()
        graph.replay()
        check()


def test_prepared_block(vq):
    """A function of the block's calls, recorded by prepare() and repeated."""
    rng = np.random.default_rng(7)
    x = gen.to_storage(rng.standard_normal((6, 256)).astype(np.float32), "bf16").to(DEV)
    w = gen.to_storage((rng.standard_normal((2 * 96, 256)) * 0.05).astype(np.float32), "bf16").to(DEV)
    wc, ws = vq.vq_pack_weights(w, 8)
    gc, gs = vq.vq_pack_weights_group(w, 64)
    off = torch.tensor([0, 4, 6], dtype=torch.int32, device=DEV)

    def f(x):
        c, s = vq.vq_rmsnorm_quant(x, None, 8, EPS)
        n = vq.vq_rmsnorm(x, None, EPS)
        return (vq.vq_qgemm_experts(c, s, wc, ws, 8, off), vq.vq_w4_gemv(n, gc, gs),
                vq.vq_gemm_dense_experts(n, w.view(2, 96, 256), off))
    launch, got = vq.prepare(f, x)
    want = f(x)
    for _ in range(2):
        for t in got:
            t.zero_()
        launch()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_one_token(vq, dt):
    rng = np.random.default_rng(11)
    k, n = 1920, 640
    x, r, wn = (gen.to_storage(rng.standard_normal((1, k)).astype(np.float32), dt) for _ in range(3))
    w = gen.to_storage((rng.standard_normal((n, k)) * 0.02).astype(np.float32), dt)
    codes, scales = vq.vq_pack_weights_group(w.to(DEV), 128)
    y, h = vq.vq_rmsnorm(x.to(DEV), wn[0].contiguous().to(DEV), EPS, residual=r.to(DEV))
    out = vq.vq_w4_gemv(y, codes, scales, torch.float32)
    torch.cuda.synchronize()
    oh, v = onorm.rows(gen.as_numpy_bits(x), dt, onum.to_f32(gen.as_numpy_bits(wn), dt)[0], EPS, gen.as_numpy_bits(r))
    ys = onum.from_f32(v, dt)
    assert np.array_equal(bits(h), oh) and np.array_equal(bits(y), ys)
    _, packed, s = group4.pack(gen.as_numpy_bits(w), dt, 128)
    ex, b = group4.exact(ys, dt, packed, s, 128)
    assert np.all(np.abs(out.cpu().numpy() - ex) <= b)
