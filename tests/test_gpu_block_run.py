"""The operators between the layers of a block as a network runs them: gated norm to codes, the
quantized projection with its requests' adapters, the norm after it, the router, the experts'
products and the way back into the residual stream, and the next norm.

Each step is held against its oracle on the step before's own outputs; the whole is captured in a
graph and replayed with other inputs, modulations, routing and adapters, and recorded by prepare().
"""
import numpy as np
import pytest
import torch

import gen
from oracle import gated as og
from oracle import lowrank as ol
from oracle import norm as onorm
from oracle import numerics as onum
from oracle import quantizer, router

pytestmark = pytest.mark.gpu

DEV = "cuda"
EPS = 1e-6
DIM, MID, E, TOP, AD, RANK = 320, 192, 6, 2, 3, 16


@pytest.fixture(scope="module")
def vq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_quantized_linear_vq_amd as m
    return m


def bits(t):
    return gen.as_numpy_bits(t.cpu().contiguous())


def f32(t):
    t = t.cpu().contiguous()
    return t.numpy() if t.dtype == torch.float32 else onum.to_f32(gen.as_numpy_bits(t), "bf16")


def half(rng, *shape, scale=1.0):
    return gen.to_storage((rng.standard_normal(shape) * scale).astype(np.float32), "bf16").to(DEV)


class Block:
    def __init__(self, vq, m, sets, seed=0):
        rng = np.random.default_rng(seed)
        self.vq, self.m, self.sets = vq, m, sets
        self.proj = half(rng, DIM, DIM, scale=0.05)
        self.up, self.down = half(rng, E * MID, DIM, scale=0.05), half(rng, E * DIM, MID, scale=0.05)
        self.pc, self.ps = vq.vq_pack_weights(self.proj, 8, kblock=True)
        self.uc, self.us = vq.vq_pack_weights(self.up, 4)
        self.dc, self.ds = vq.vq_pack_weights(self.down, 8)
        self.router = half(rng, E, DIM, scale=0.1)
        self.ad_down, self.ad_up = half(rng, AD, RANK, DIM, scale=0.05), half(rng, AD, DIM, RANK, scale=0.1)
        self.w = torch.from_numpy((1 + 0.1 * rng.standard_normal(DIM)).astype(np.float32)).to(DEV)
        self.bias = torch.from_numpy((0.1 * rng.standard_normal(E)).astype(np.float32)).to(DEV)
        self.h, self.y = half(rng, m, DIM, scale=2.0), half(rng, m, DIM)
        self.mod = torch.zeros(sets, 6 * DIM, device=DEV)
        self.index = torch.zeros(m, dtype=torch.int32, device=DEV)
        self.adapter = torch.zeros(m, dtype=torch.int32, device=DEV)
        self.new_inputs(seed)

    def new_inputs(self, seed):
        rng = np.random.default_rng([seed, 1])
        self.h.copy_(half(rng, self.m, DIM, scale=2.0))
        self.y.copy_(half(rng, self.m, DIM))
        self.mod.copy_(torch.from_numpy((0.4 * rng.standard_normal((self.sets, 6 * DIM))).astype(np.float32)))
        self.index.copy_(torch.from_numpy(rng.integers(0, self.sets, self.m).astype(np.int32)))
        self.adapter.copy_(torch.from_numpy(rng.integers(-1, AD, self.m).astype(np.int32)))

    def part(self, i):
        return self.mod[:, i * DIM:(i + 1) * DIM]

    def run(self):
        vq, p = self.vq, self.part
        c, s, h1 = vq.vq_gated_norm_quant(self.y, self.h, 8, norm="layer", gate=p(0), mod_scale=p(1), mod_shift=p(2),
                                          index=self.index, post="rms", post_weight=self.w)
        a, _ = vq.vq_gated_norm(None, h1, norm="layer", mod_scale=p(1), mod_shift=p(2), index=self.index)
        y1 = vq.vq_qgemm_dequant(c, s, self.pc, self.ps, 8)
        y2 = vq.vq_lowrank_add(y1, a, self.ad_down, self.ad_up, self.adapter)
        n, h2 = vq.vq_gated_norm(y2, h1, weight=self.w, gate=p(3), index=self.index)
        logits = vq.vq_gemm_dense(n, self.router, torch.float32)
        off, rows, wt, ch, place = vq.vq_route_experts(logits, TOP, score="sigmoid", bias=self.bias, groups=3, top_groups=2)
        c2, s2 = vq.vq_quant_act(n, 8, "token")
        mid = vq.vq_qgemm_experts(c2, s2, self.uc, self.us, 4, off, rows=rows)
        c3, s3 = vq.vq_quant_act(mid, 8, "token")
        y3 = vq.vq_qgemm_experts(c3, s3, self.dc, self.ds, 8, off)
        h3 = vq.vq_combine_experts(y3, place, wt, residual=h2, gate=p(4), index=self.index)
        return dict(c=c, s=s, h1=h1, a=a, y1=y1, y2=y2, n=n, h2=h2, logits=logits, off=off, rows=rows, wt=wt, ch=ch, place=place,
                    c2=c2, s2=s2, mid=mid, y3=y3, h3=h3)

    def check(self, o):
        torch.cuda.synchronize()
        mod, idx, w = self.mod.cpu().numpy(), self.index.cpu().numpy(), self.w.cpu().numpy()

        def p(i):
            return mod[:, i * DIM:(i + 1) * DIM]
        s1, v = og.rows(bits(self.y), bits(self.h), "bf16", "layer", None, EPS, "rms", w, 1.0, p(0), p(1), p(2), idx)
        oc, osc = onorm.quant(v, 8)
        assert np.array_equal(bits(o["h1"]), s1) and np.array_equal(o["c"].cpu().numpy(), oc) and np.array_equal(f32(o["s"]), osc)
        assert np.array_equal(bits(o["a"]), onum.from_f32(v, "bf16"))
        delta, bound = ol.exact(f32(o["a"]).astype(np.float64), f32(self.ad_down).astype(np.float64), f32(self.ad_up).astype(np.float64),
                                self.adapter.cpu().numpy())
        want = f32(o["y1"]) + delta
        bound += 2.0 ** -24 * (np.abs(want) + bound)
        assert np.all(np.abs(f32(o["y2"]) - want) <= bound + 2.0 ** -8 * (np.abs(want) + bound))
        s2, v = og.rows(bits(o["y2"]), bits(o["h1"]), "bf16", "rms", w, EPS, gate=p(3), index=idx)
        assert np.array_equal(bits(o["h2"]), s2) and np.array_equal(bits(o["n"]), onum.from_f32(v, "bf16"))
        off, rows, wt, ch, place = router.route(f32(o["logits"]).astype(np.float64), TOP, score="sigmoid", bias=self.bias.cpu().numpy().astype(np.float64),
                                                groups=3, keep=2)
        for got, exp in ((o["off"], off), (o["rows"], rows), (o["ch"], ch), (o["place"], place)):
            assert np.array_equal(got.cpu().numpy(), exp)
        assert np.all(np.abs(f32(o["wt"]) - wt) <= (2.0 ** -24 + 2.0 ** -40) * wt)
        # the experts' products equal the single layer's rows, exact integers and one rounding
        codes = quantizer.pack_weights(bits(self.up), "bf16", 4)
        acc = np.stack([o["c2"].cpu().numpy()[t].astype(np.int64) @ codes[0][e * MID:(e + 1) * MID].astype(np.int64).T
                        for e in range(E) for t in rows[off[e]:off[e + 1]]])
        exp_of = np.repeat(np.arange(E), np.diff(off))
        sc = (f32(o["s2"])[rows[:len(exp_of)]][:, None] * codes[2].reshape(E, MID)[exp_of]).astype(np.float32)
        assert np.array_equal(bits(o["mid"])[:len(acc)], onum.from_f32((acc.astype(np.float32) * sc).astype(np.float32), "bf16"))
        h3 = router.combine(f32(o["y3"]), place, f32(o["wt"]), f32(o["h2"]), p(4), idx)
        assert np.array_equal(bits(o["h3"]), onum.from_f32(h3, "bf16"))


@pytest.mark.parametrize("m,sets", [(1, 1), (5, 3), (90, 4), (1300, 7)])
def test_block(vq, m, sets):
    b = Block(vq, m, sets, seed=m)
    b.check(b.run())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        b.run()
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            out = b.run()
    torch.cuda.synchronize()
    for seed in (2, 3, 4):
        b.new_inputs(seed)
        for t in out.values():
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        b.check(out)
        want = b.run()
        torch.cuda.synchronize()
        assert all(torch.equal(out[k], want[k]) for k in want)


def test_prepared_block(vq):
    b = Block(vq, 40, 4)
    launch, out = vq.prepare(b.run)
    others = [torch.full((n,), 7, dtype=torch.uint8, device=DEV) for n in (64, 40 * 640, 40 * 320, 80 * 384, 1024) for _ in range(30)]
    for seed in (5, 6):
        b.new_inputs(seed)
        for t in out.values():
            t.zero_()
        launch()
        b.check(out)
    assert all(bool((t == 7).all()) for t in others)


def test_two_streams_at_once(vq):
    """Calls on two streams share nothing but their weights."""
    blocks = [Block(vq, m, 4, seed=m) for m in (300, 700)]
    want = [b.run() for b in blocks]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in blocks]
    got = [None, None]
    for _ in range(3):
        for i, (b, s) in enumerate(zip(blocks, streams)):
            with torch.cuda.stream(s):
                got[i] = b.run()
        torch.cuda.synchronize()
        for w, g in zip(want, got):
            assert all(torch.equal(w[k], g[k]) for k in w)


@pytest.mark.parametrize("branch,k", [(True, 1920), (False, 12288), (True, 4095)])
def test_norms_of_calls_larger_than_the_cache(vq, branch, k):
    """They equal those of the rows in pieces."""
    m = (200 << 20) // (k * (8 if branch else 4)) + 1100
    g = torch.Generator(device=DEV).manual_seed(k)
    h = torch.randn(m, k, device=DEV, generator=g).bfloat16()
    y = torch.randn(m, k, device=DEV, generator=g).bfloat16() if branch else None
    mod = torch.randn(3, k, device=DEV, generator=g)
    index = torch.randint(0, 3, (m,), device=DEV, generator=g, dtype=torch.int32)
    how = dict(norm="layer", mod_scale=mod, index=index, **(dict(gate=mod, post="rms") if branch else {}))
    n, s = vq.vq_gated_norm(y, h, **how)
    quant = vq.vq_gated_norm_quant(y, h, 8, **how) if k % 64 == 0 else None
    torch.cuda.synchronize()
    for lo in range(0, m, 7001):
        at = slice(lo, lo + 7001)
        part = dict(how, index=index[at])
        n2, s2 = vq.vq_gated_norm(None if y is None else y[at], h[at], **part)
        assert torch.equal(n[at], n2) and torch.equal(s[at], s2)
        if quant:
            for a, b in zip(quant, vq.vq_gated_norm_quant(None if y is None else y[at], h[at], 8, **part)):
                assert torch.equal(a[at], b)
