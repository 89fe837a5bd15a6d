"""GPU parity of the routing to experts and of the experts' rows back to their tokens
(oracle/router.py).

Choices, places, offsets and rows are whole numbers and must equal the oracle's.  Weights are
float64 values rounded once: a float64 value that is off by E 2^-50 of itself moves the rounded one by at most
that and the rounding, 2^-24.  The denominator of a softmax that is not renormalised, chosen by the scores,
is a float64 sum of positive terms that are each within 2^-22 (the hardware's 2^f within an ulp, 2^-23, of a
fraction rounded to 2^-26 of 1, ln 2 2^-26 of the term), so it is within 2^-22 too.  Combined rows are float32 operations in one order: bit for bit.
"""
import numpy as np
import pytest
import torch

import gen
from oracle import numerics as onum
from oracle import router

pytestmark = pytest.mark.gpu

DEV = "cuda"
TD = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def vq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_quantized_linear_vq_amd as m
    return m


def scores(m, e, dt, masked=0.0, seed=0):
    rng = np.random.default_rng([m, e, seed])
    x = (1.5 * rng.standard_normal((m, e))).astype(np.float32)
    x[rng.random((m, e)) < masked] = -np.inf
    x[rng.random(m) < masked / 2] = -np.inf
    return torch.from_numpy(x).to(TD[dt])


def check(got, x, top, bias=None, **how):
    torch.cuda.synchronize()
    off, rows, w, ch, place = (t.cpu().numpy() for t in got)
    how = {{"top_groups": "keep", "group_best": "best"}.get(k, k): v for k, v in how.items()}
    want = router.route(x.double().cpu().numpy(), top, bias=None if bias is None else bias.double().cpu().numpy(), **how)
    assert np.array_equal(ch, want[3])
    assert np.array_equal(off, want[0]) and np.array_equal(rows, want[1]) and np.array_equal(place, want[4])
    assert np.array_equal(np.isnan(w), np.isnan(want[2]))
    ok = ~np.isnan(w)
    summed = 0.0 if how.get("renorm", True) or how.get("score", "softmax") == "sigmoid" else 2.0 ** -22 + 2.0 ** -40
    rel = 2.0 ** -24 + x.shape[1] * 2.0 ** -50 + summed
    assert np.all(np.abs(w[ok].astype(np.float64) - want[2][ok]) <= rel * np.abs(want[2][ok]) + 2.0 ** -150)


@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("m,e,top,how,masked", [
    (1, 1, 1, {}, 0.0), (1, 16, 2, {}, 0.0), (3, 7, 7, dict(score="sigmoid", renorm=False), 0.3), (65, 17, 3, {}, 0.1),
    (5, 64, 8, dict(score="sigmoid", bias=True, groups=8, top_groups=4, group_best=2), 0.0),
    (64, 96, 4, dict(score="sigmoid", bias=True, groups=6, top_groups=3, group_best=2), 0.2),
    (130, 160, 6, dict(renorm=False, scale=2.5), 0.02), (63, 256, 8, dict(groups=8, top_groups=3), 0.0),
    (40, 257, 5, dict(bias=True), 0.1), (33, 1024, 32, dict(score="sigmoid", bias=True, groups=64, top_groups=9, group_best=2), 0.5),
    (20, 513, 32, {}, 0.9), (70, 30, 3, dict(groups=10, top_groups=2, group_best=2), 0.4),
    (30, 128, 32, dict(bias=True, groups=32, top_groups=8, group_best=1), 0.1), (257, 33, 1, dict(bias=True, renorm=False), 0.0),
    (300, 12, 5, dict(groups=6, top_groups=6, group_best=2, bias=True), 0.5),
])
def test_routing_equals_the_definition(vq, m, e, top, how, masked, dt):
    x = scores(m, e, dt, masked)
    how = dict(how)
    bias = None
    if how.pop("bias", False):
        bias = torch.from_numpy((0.1 * np.random.default_rng(e).standard_normal(e)).astype(np.float32))
    got = vq.vq_route_experts(x.to(DEV), top, bias=None if bias is None else bias.to(DEV), **how)
    check(got, x, top, bias, **how)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("how", [dict(), dict(groups=4, top_groups=2), dict(groups=4, top_groups=2, group_best=2)])
def test_ties_go_to_the_lower_index(vq, score, how):
    x = torch.from_numpy(np.random.default_rng(1).integers(-1, 2, (200, 32)).astype(np.float32))
    x[0] = 0.0
    check(vq.vq_route_experts(x.to(DEV), 6, score=score, **how), x, 6, score=score, **how)
    bias = torch.zeros(32)
    check(vq.vq_route_experts(x.to(DEV), 6, score=score, bias=bias.to(DEV), **how), x, 6, bias, score=score, **how)


def test_scores_whose_p_is_the_same_number(vq):
    x = torch.full((4, 20), -3e38)
    x[0, 5:9] = torch.tensor([50.0, 60.0, 40.0, 55.0])
    x[1] = torch.arange(20) - 2000.0
    x[1, 3] = 0.0
    x[2, 7] = -2e38
    for score in ("softmax", "sigmoid"):
        check(vq.vq_route_experts(x.to(DEV), 5, score=score), x, 5, score=score)
    low = x.clamp(min=-65504).half()
    check(vq.vq_route_experts(low.to(DEV), 5), low, 5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 5])
def test_rows_and_biases_that_are_not_finite(vq, score, groups):
    inf, nan = float("inf"), float("nan")
    x = scores(12, 40, "fp32")
    x[1, 3], x[2, 39], x[3], x[4, :39], x[5, 7], x[6] = nan, inf, -inf, -inf, -inf, nan
    how = dict(score=score, groups=groups, top_groups=max(1, groups - 2))
    check(vq.vq_route_experts(x.to(DEV), 4, **how), x, 4, **how)
    for v in (-inf, inf, nan):
        bias = torch.zeros(40)
        bias[11] = v
        check(vq.vq_route_experts(x.to(DEV), 4, bias=bias.to(DEV), **how), x, 4, bias, **how)


@pytest.mark.parametrize("m,e,top", [(4096, 8, 2), (1000, 1024, 7), (17776, 160, 6), (5000, 1, 1), (100003, 9, 8), (30000, 300, 32)])
def test_many_rows_keep_their_order(vq, m, e, top):
    """Places are a permutation, sorted by expert and, in an expert, by token."""
    x = scores(m, e, "fp32", 0.05)
    off, rows, w, ch, place = vq.vq_route_experts(x.to(DEV), top)
    torch.cuda.synchronize()
    order = torch.sort(torch.where(x == -np.inf, -np.inf, x), dim=1, descending=True, stable=True)
    want = torch.where(order.values[:, :top] == -np.inf, -1, order.indices[:, :top])
    assert torch.equal(ch.cpu().long(), want)
    flat = torch.where(want < 0, e, want).flatten()
    at = torch.sort(flat, stable=True).indices
    n = int((flat < e).sum())
    assert torch.equal(off.cpu().long(), torch.searchsorted(flat[at].contiguous(), torch.arange(e + 1)))
    assert torch.equal(rows.cpu()[:n].long(), at[:n] // top) and bool((rows[n:] == -1).all())
    where = torch.full((m * top,), -1)
    where[at[:n]] = torch.arange(n)
    assert torch.equal(place.cpu().flatten().long(), where)


@pytest.mark.parametrize("m", [1, 4, 5, 16, 17, 64, 65, 300])
@pytest.mark.parametrize("e,groups", [(64, 8), (65, 5), (256, 16), (257, 1), (360, 12), (512, 64), (1024, 64), (1023, 3)])
def test_every_way_of_cutting_the_rows(vq, m, e, groups):
    x = scores(m, e, "fp32", 0.3)
    bias = 0.05 * torch.randn(e, generator=torch.Generator().manual_seed(e))
    how = dict(score="sigmoid", groups=groups, top_groups=max(1, groups // 3), group_best=2)
    top = min(8, e // groups * how["top_groups"])
    check(vq.vq_route_experts(x.to(DEV), top, bias=bias.to(DEV), **how), x, top, bias, **how)


def test_no_tokens(vq):
    off, rows, w, ch, place = vq.vq_route_experts(torch.empty(0, 9, device=DEV), 3)
    torch.cuda.synchronize()
    assert off.tolist() == [0] * 10 and rows.numel() == 0 and place.shape == (0, 3)
    assert vq.vq_combine_experts(torch.empty(0, 8, device=DEV), place, w).shape == (0, 8)


def test_padded_rows_of_scores_and_given_outputs(vq):
    wide = torch.full((50, 40), float("nan"), dtype=torch.bfloat16, device=DEV)
    wide[:, :24] = scores(50, 24, "bf16").to(DEV)
    want = vq.vq_route_experts(wide[:, :24].contiguous(), 4)
    outs = dict(zip(("offsets", "rows", "weights", "experts", "place"), (torch.empty_like(t) for t in want)))
    ws = torch.full((vq.vq_route_experts_workspace_elems(50, 24) + 8,), 77, dtype=torch.int32, device=DEV)
    got = vq.vq_route_experts(wide[:, :24], 4, ws=ws, **outs)
    assert all(g is o for g, o in zip(got, outs.values())) and all(torch.equal(a, b) for a, b in zip(got, want))
    assert bool((ws[-8:] == 77).all())


def test_routing_in_a_replayed_graph(vq):
    m, e, top = 500, 48, 4
    x = scores(m, e, "fp32").to(DEV)
    outs = [torch.empty_like(t) for t in vq.vq_route_experts(x, top)]
    names = ("offsets", "rows", "weights", "experts", "place")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            vq.vq_route_experts(x, top, **dict(zip(names, outs)))
    for i in range(3):
        x.copy_(scores(m, e, "fp32", 0.1 * i, seed=i))
        for t in outs:
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        want = vq.vq_route_experts(x, top)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


# ------------------------------------------------------------------ the way back

def rows_of(t, dt):
    return t.numpy() if dt == "fp32" else onum.to_f32(gen.as_numpy_bits(t), dt)


def bits(a):
    a = gen.as_numpy_bits(a.cpu().contiguous()) if isinstance(a, torch.Tensor) and a.element_size() == 2 else a
    a = a.cpu().numpy() if isinstance(a, torch.Tensor) else a
    a = np.ascontiguousarray(a)
    return a.view({2: np.uint16, 4: np.uint32}[a.dtype.itemsize])


@pytest.mark.parametrize("ydt,odt", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "fp32"), ("fp16", "fp32"), ("fp32", "bf16"),
                                     ("fp32", "fp16"), ("fp32", "fp32")])
@pytest.mark.parametrize("m,n,top,res,sets,g32", [
    (1, 1, 1, False, 0, True), (3, 7, 2, True, 3, True), (8, 1920, 2, True, 8, False), (70, 2047, 4, True, 0, True),
    (33, 513, 32, False, 1, False), (40, 64, 3, True, -6, True), (25, 4096, 8, False, -3, False), (300, 100, 2, True, 10, True),
])
def test_combining_equals_the_definition(vq, m, n, top, res, sets, g32, ydt, odt):
    rng = np.random.default_rng([m, n, top])
    t = m * top + 3

    def make(dt, *shape):
        return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(TD[dt])
    y = make(ydt, t, n)
    place = rng.permutation(t)[:m * top].reshape(m, top).astype(np.int32)
    w = rng.random((m, top)).astype(np.float32)
    gone = rng.random((m, top)) < 0.2
    y[torch.from_numpy(place[gone]).long()] = float("nan")
    place[gone], w[gone] = -1, 0.0
    r = make(odt, m, n) if res else None
    gdt = "fp32" if g32 or (ydt == odt == "fp32") else ydt if ydt != "fp32" else odt
    gate = make(gdt, abs(sets), n) if sets else None
    index = torch.from_numpy(rng.integers(-1, -sets + 1, m).astype(np.int32)) if sets < 0 else None
    got = vq.vq_combine_experts(y.to(DEV), torch.from_numpy(place).to(DEV), torch.from_numpy(w).to(DEV),
                                residual=None if r is None else r.to(DEV), gate=None if gate is None else gate.to(DEV),
                                index=None if index is None else index.to(DEV), out_dtype=TD[odt])
    torch.cuda.synchronize()
    at = None if gate is None else np.arange(m) // (m // sets) if index is None else index.numpy()
    want = router.combine(rows_of(y, ydt), place, w, None if r is None else rows_of(r, odt), None if gate is None else rows_of(gate, gdt), at)
    assert got.dtype == TD[odt]
    assert np.array_equal(bits(got), bits(want if odt == "fp32" else onum.from_f32(want, odt)))


def test_places_outside_the_rows_and_weights_that_are_nan(vq):
    y = torch.ones(6, 24, dtype=torch.bfloat16, device=DEV)
    place = torch.tensor([[0, 6], [-5, 2 ** 31 - 1], [1, -1], [2, 3]], dtype=torch.int32, device=DEV)
    w = torch.tensor([[1.0, 2.0], [3.0, 4.0], [1.0, float("nan")], [1.0, 1.0]], device=DEV)
    out = vq.vq_combine_experts(y, place, w).float().cpu()
    assert bool((out[0] == 1).all() and (out[1] == 0).all() and out[2].isnan().all() and (out[3] == 2).all())


@pytest.mark.parametrize("n,pad", [(1920, 0), (1921, 0), (512, 3), (7, 1)])
def test_residual_in_place_and_pitches(vq, n, pad):
    m, top = 37, 3
    g = torch.Generator(device=DEV).manual_seed(3)

    def wide(rows):
        return torch.randn(rows, n + pad, device=DEV, generator=g).bfloat16()[:, :n]
    y, r = wide(m * top), wide(m)
    place = torch.randperm(m * top, device=DEV, generator=g).int().view(m, top)
    w = torch.rand(m, top, device=DEV, generator=g)
    gate = wide(m)
    want = vq.vq_combine_experts(y.contiguous(), place, w, residual=r.contiguous(), gate=gate.contiguous())
    assert torch.equal(vq.vq_combine_experts(y, place, w, residual=r, gate=gate), want)
    base = torch.full((m, n + pad + 2), 5.0, dtype=torch.bfloat16, device=DEV)
    base[:, 1:n + 1] = r
    got = vq.vq_combine_experts(y, place, w, residual=base[:, 1:n + 1], gate=gate, out=base[:, 1:n + 1])
    assert torch.equal(got, want) and bool((base[:, 0] == 5).all() and (base[:, n + 1:] == 5).all())


@pytest.mark.parametrize("w_bits", [8, 4])
def test_a_feed_forward_over_experts(vq, w_bits):
    """Router, product over experts and the way back, against each token through its own experts."""
    m, e, top, dim, n = 150, 12, 3, 256, 192
    g = torch.Generator(device=DEV).manual_seed(9)
    x = torch.randn(m, dim, device=DEV, generator=g).bfloat16()
    w = (0.1 * torch.randn(e * n, dim, device=DEV, generator=g)).bfloat16()
    logits = torch.randn(m, e, device=DEV, generator=g)
    logits[7] = -float("inf")
    logits[8, 1:] = -float("inf")
    res = torch.randn(m, n, device=DEV, generator=g).bfloat16()
    wc, ws = vq.vq_pack_weights(w, w_bits, kblock=True)
    c, s = vq.vq_quant_act(x, 8, "token")
    off, rows, p, ch, place = vq.vq_route_experts(logits, top)
    y = vq.vq_qgemm_experts(c, s, wc, ws, w_bits, off, rows=rows, out_dtype=torch.float32)
    out = vq.vq_combine_experts(y, place, p, residual=res)
    torch.cuda.synchronize()
    each = torch.stack([vq.vq_qgemm_dequant(c, s, wc[:, i * n:(i + 1) * n].contiguous(), ws[i * n:(i + 1) * n].contiguous(), w_bits,
                                            out_dtype=torch.float32) for i in range(e)]).cpu().numpy()
    pn, cn = p.cpu().numpy(), ch.cpu().numpy()
    want = np.zeros((m, n), np.float32)
    for j in range(top):
        q = np.where((cn[:, j] >= 0)[:, None], each[np.maximum(cn[:, j], 0), np.arange(m)], np.float32(0))
        want = (want + (q * pn[:, j][:, None]).astype(np.float32)).astype(np.float32)
    want = (want + onum.to_f32(gen.as_numpy_bits(res.cpu()), "bf16")).astype(np.float32)
    assert np.array_equal(bits(out), bits(onum.from_f32(want, "bf16")))
    assert cn[7].tolist() == [-1, -1, -1] and cn[8].tolist() == [0, -1, -1] and pn[8, 0] == 1.0
