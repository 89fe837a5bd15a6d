"""GPU parity of the low-rank adapters beside a shared projection (oracle/lowrank.py): within the
bound that its float32 sums and the two pieces of t allow, and half a step of the output's type.
"""
import numpy as np
import pytest
import torch

import gen
from oracle import lowrank as ol
from oracle import numerics as onum

pytestmark = pytest.mark.gpu

DEV = "cuda"
TD = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
# half a step of a rounding, relative, and the smallest step's half
HALF = {"bf16": (2.0 ** -8, 2.0 ** -134), "fp16": (2.0 ** -11, 2.0 ** -25), "fp32": (2.0 ** -24, 2.0 ** -150)}


@pytest.fixture(scope="module")
def vq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_quantized_linear_vq_amd as m
    return m


def f64(t, dt):
    return (t.numpy() if dt == "fp32" else onum.to_f32(gen.as_numpy_bits(t), dt)).astype(np.float64)


def make(m, n, k, r, adapters, dt, odt, index, seed=0):
    rng = np.random.default_rng([m, n, k, r, seed])

    def half(shape, scale, d=dt):
        a = (scale * rng.standard_normal(shape)).astype(np.float32)
        return torch.from_numpy(a) if d == "fp32" else gen.to_storage(a, d)
    if index == "one":
        idx = np.full(m, adapters - 1)
    elif index == "any":
        idx = rng.integers(-1, adapters + 1, m)
    elif index == "none":
        idx = np.where(rng.random(m) < 0.5, -1, adapters)
    else:  # sequences one after the other
        idx = np.sort(rng.integers(0, 5, m))
        idx = rng.integers(-1, adapters, 5)[idx]
    return dict(base=half((m, n), 1.0, odt), x=half((m, k), 1.0), down=half((adapters, r, k), k ** -0.5),
                up=half((adapters, n, r), 0.5 * r ** -0.5), index=torch.from_numpy(idx.astype(np.int32)),
                scales=torch.from_numpy((0.5 + rng.random(adapters)).astype(np.float32)))


def on(c, **kw):
    return {**{k: None if v is None else v.to(DEV) for k, v in c.items()}, **kw}


def check(got, c, dt, odt):
    torch.cuda.synchronize()
    idx = c["index"].numpy()
    with np.errstate(invalid="ignore"):
        delta, bound = ol.exact(f64(c["x"], dt), f64(c["down"], dt), f64(c["up"], dt), idx, None if c["scales"] is None else c["scales"].numpy(), dt)
    base = f64(c["base"], odt)
    g = f64(got.cpu().contiguous(), odt)
    want = base + delta
    rel, tiny = HALF[odt]
    bound = bound + 2.0 ** -24 * (np.abs(base) + np.abs(delta) + bound)  # the float32 addition
    finite = np.isfinite(want)  # an infinite x (a loud row in fp16) has outputs that are none
    assert not np.isfinite(g[~finite]).any()
    assert np.all((np.abs(g - want) <= bound + rel * (np.abs(want) + bound) + tiny)[finite])
    none = (idx < 0) | (idx >= len(c["down"]))
    assert np.array_equal(g[none], base[none])


SHAPES = [
    (1, 1, 64, 8, 1, "one"), (1, 5760, 1920, 64, 4, "one"), (3, 33, 128, 24, 2, "any"), (16, 100, 256, 16, 16, "any"),
    (17, 65, 192, 40, 5, "any"), (48, 515, 1024, 16, 12, "any"), (50, 64, 64, 128, 3, "sorted"), (200, 1000, 640, 32, 40, "any"),
    (130, 257, 4096, 104, 7, "sorted"), (1024, 320, 128, 8, 6, "sorted"), (1100, 129, 320, 128, 9, "any"),
    (1030, 1030, 64, 72, 3, "sorted"), (64, 40, 512, 32, 2, "none"), (8200, 40, 256, 32, 5, "sorted"), (8197, 24, 128, 56, 30, "any"),
    (8300, 17, 192, 120, 4, "sorted"), (300, 130, 256, 48, 4, "sorted"), (100, 64, 9088, 64, 2, "any"), (65, 33, 8256, 8, 3, "any"),
    (5200, 19, 4160, 16, 4, "sorted"), (1023, 70, 64, 24, 3, "any"), (8300, 1100, 64, 104, 9, "any"), (8200, 1283, 128, 40, 4, "sorted"),
]


@pytest.mark.parametrize("dt,odt", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "fp32"), ("fp16", "fp32")])
@pytest.mark.parametrize("m,n,k,r,adapters,index", SHAPES)
def test_within_the_bound(vq, m, n, k, r, adapters, index, dt, odt):
    c = make(m, n, k, r, adapters, dt, odt, index)
    check(vq.vq_lowrank_add(**on(c)), c, dt, odt)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("m", [5, 1500])
def test_whole_numbers_are_exact(vq, m, dt):
    """Sums below 2^24 of whole numbers, and t of at most 16 bits: nothing is rounded."""
    rng = np.random.default_rng(m)
    k, r, n, ad = 256, 24, 72, 6

    def whole(*shape, big):
        return gen.to_storage(rng.integers(-big, big + 1, shape).astype(np.float32), dt)
    c = dict(base=torch.from_numpy(rng.integers(-99, 100, (m, n)).astype(np.float32)), x=whole(m, k, big=4), down=whole(ad, r, k, big=3),
             up=whole(ad, n, r, big=5), index=torch.from_numpy(rng.integers(-1, ad, m).astype(np.int32)),
             scales=torch.from_numpy(2.0 ** rng.integers(0, 4, ad).astype(np.float32)))
    got = vq.vq_lowrank_add(**on(c))
    torch.cuda.synchronize()
    delta, _ = ol.exact(f64(c["x"], dt), f64(c["down"], dt), f64(c["up"], dt), c["index"].numpy(), c["scales"].numpy(), dt)
    assert np.array_equal(got.cpu().numpy().astype(np.float64), f64(c["base"], "fp32") + delta)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("size", [1e-3, 3e3, 3e4])
def test_loud_and_quiet_rows(vq, dt, size):
    """t far beyond fp16's range, beside rows of another size."""
    c = make(40, 96, 512, 16, 3, dt, "fp32", "any")
    c["x"] = (c["x"].float() * torch.where(torch.arange(40) % 3 == 0, size, 1.0)[:, None]).to(TD[dt])
    c["scales"] = c["scales"] * 100.0
    check(vq.vq_lowrank_add(**on(c)), c, dt, "fp32")


@pytest.mark.parametrize("m", [40, 1100])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("size", [1e33, 1e-30])
def test_scales_at_the_ends_of_float32(vq, dt, size, m):
    c = make(m, 96, 512, 16, 3, dt, "fp32", "any")
    c["base"] = c["base"] * size
    c["scales"] = c["scales"] * size
    check(vq.vq_lowrank_add(**on(c)), c, dt, "fp32")


def test_without_scales(vq):
    c = make(20, 64, 128, 8, 3, "bf16", "bf16", "any")
    c["scales"] = None
    check(vq.vq_lowrank_add(**on(c)), c, "bf16", "bf16")


@pytest.mark.parametrize("m", [30, 1200])
@pytest.mark.parametrize("what", ["x", "down", "up", "scales"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_what_is_not_finite_stays_in_its_rows(vq, m, what, value):
    c = make(m, 80, 128, 16, 4, "bf16", "bf16", "any")
    idx = c["index"].numpy()
    good = vq.vq_lowrank_add(**on(c))
    if what == "x":
        row = int(np.nonzero(idx == 2)[0][0])
        c["x"][row, 5] = value
        bad = np.arange(m) == row
    else:
        c[what][(2,) + (3,) * (c[what].dim() - 1)] = value
        bad = idx == 2
    got = vq.vq_lowrank_add(**on(c))
    torch.cuda.synchronize()
    bad = torch.from_numpy(bad).to(DEV)
    assert torch.equal(got[~bad], good[~bad])
    assert bool((~got[bad].float().isfinite()).any(1).all())


def test_rows_without_an_adapter_keep_their_bits(vq):
    c = make(40, 50, 128, 8, 2, "fp16", "fp16", "none")
    c["base"][3] = float("nan")
    c["base"][4] = float("-inf")
    c["x"][:] = float("nan")
    got = vq.vq_lowrank_add(**on(c))
    torch.cuda.synchronize()
    assert np.array_equal(gen.as_numpy_bits(got.cpu()).view(np.uint16), gen.as_numpy_bits(c["base"]).view(np.uint16))


@pytest.mark.parametrize("m", [9, 1030])
def test_in_place_pitches_and_rows_behind(vq, m):
    n, k = 77, 128
    c = on(make(m, n, k, 16, 3, "bf16", "bf16", "any"))
    want = vq.vq_lowrank_add(**c)
    wide = torch.full((m + 2, n + 5), 3.0, dtype=torch.bfloat16, device=DEV)
    wide[1:m + 1, 3:n + 3] = c["base"]
    xw = torch.full((m, k + 8), float("nan"), dtype=torch.bfloat16, device=DEV)
    xw[:, :k] = c["x"]
    got = vq.vq_lowrank_add(**{**c, "base": wide[1:m + 1, 3:n + 3], "x": xw[:, :k], "out": wide[1:m + 1, 3:n + 3]})
    assert torch.equal(got, want)
    wide[1:m + 1, 3:n + 3] = 3.0
    assert bool((wide == 3.0).all())
    need = vq.vq_lowrank_workspace_elems(m, 3, 16, k)
    ws = torch.full((need + 64,), 9.0, device=DEV)
    assert torch.equal(vq.vq_lowrank_add(**c, ws=ws), want) and bool((ws[need:] == 9.0).all())


def test_no_rows(vq):
    c = make(0, 16, 64, 8, 2, "bf16", "bf16", "one")
    assert vq.vq_lowrank_add(**on(c)).shape == (0, 16)


@pytest.mark.parametrize("m", [33, 2000])
def test_replayed_with_another_index(vq, m):
    c = on(make(m, 200, 256, 32, 6, "fp16", "fp16", "any"))
    out = torch.empty_like(c["base"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            vq.vq_lowrank_add(**c, out=out)
    for i in range(3):
        c["index"].copy_(torch.randint(-1, 7, (m,), device=DEV) if i else torch.full((m,), 4, device=DEV))
        c["x"].copy_(torch.randn_like(c["x"]))
        out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        want = vq.vq_lowrank_add(**c)
        torch.cuda.synchronize()
        assert torch.equal(out, want)


@pytest.mark.parametrize("rows", [7, 1300])
def test_beside_the_quantized_projection(vq, rows):
    """The layer's product with its adapters, and the same with the adapters merged by hand in float64."""
    g = torch.Generator(device=DEV).manual_seed(5)
    k, n, r, ad = 256, 320, 16, 5
    x = torch.randn(rows, k, device=DEV, generator=g).bfloat16()
    w = (0.1 * torch.randn(n, k, device=DEV, generator=g)).bfloat16()
    down = (torch.randn(ad, r, k, device=DEV, generator=g) / 16).bfloat16()
    up = (0.2 * torch.randn(ad, n, r, device=DEV, generator=g)).bfloat16()
    index = torch.randint(-1, ad, (rows,), device=DEV, generator=g, dtype=torch.int32)
    wc, ws = vq.vq_pack_weights(w, 8, kblock=True)
    codes, sa = vq.vq_quant_act(x, 8, "token")
    base = vq.vq_qgemm_dequant(codes, sa, wc, ws, 8, out_dtype=torch.float32)
    got = vq.vq_lowrank_add(base, x, down, up, index)
    torch.cuda.synchronize()
    c = dict(base=base.cpu(), x=x.cpu(), down=down.cpu(), up=up.cpu(), index=index.cpu(), scales=None)
    check(got, c, "bf16", "fp32")
