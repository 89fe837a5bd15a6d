"""GPU parity of the norms before and after a block with its gate and residual scale, as 16-bit
rows and as activation codes (oracle/gated.py).

Moments are float64 on both sides and every later step is one float32 operation or one
rounding, so sums, outputs, codes and scales must equal the oracle's bit for bit.
"""
import numpy as np
import pytest
import torch

import gen
from oracle import gated as og
from oracle import norm as onorm
from oracle import numerics as onum

pytestmark = pytest.mark.gpu

DEV = "cuda"
EPS = 1e-6


@pytest.fixture(scope="module")
def vq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_quantized_linear_vq_amd as m
    return m


def bits(t):
    a = gen.as_numpy_bits(t.cpu().contiguous()) if isinstance(t, torch.Tensor) else np.ascontiguousarray(t)
    return a.view(np.uint16 if a.dtype.itemsize == 2 else np.uint32 if a.dtype.itemsize == 4 else a.dtype)


def f32(t, dt):
    return t.numpy() if t.dtype == torch.float32 else onum.to_f32(gen.as_numpy_bits(t), dt)


class Case:
    """Operands on both sides.  mods: which of gate (g), scale (c) and shift (d) there are; w, pw: "none",
    "same" or "f32"; index: None, "any" (some outside the sets) or "sorted"."""

    def __init__(self, m, k, dt, branch=True, post=None, norm="rms", mods="gcd", sets=1, index=None, mod32=False, w="none",
                 pw="none", alpha=1.0, seed=0):
        rng = np.random.default_rng([m, k, sets, seed])

        def half(*shape, scale=1.0, mean=0.0):
            return gen.to_storage((mean + scale * rng.standard_normal(shape)).astype(np.float32), dt)

        def weight(kind):
            v = (1 + 0.2 * rng.standard_normal(k)).astype(np.float32)
            return None if kind == "none" else torch.from_numpy(v) if kind == "f32" else gen.to_storage(v, dt)
        self.dt, self.norm, self.alpha = dt, norm, alpha
        self.y = half(m, k, scale=3.0) if branch else None
        self.h = half(m, k, scale=2.0, mean=0.5)
        self.post = post if branch else None
        self.w, self.pw = weight(w), weight(pw) if self.post else None
        t = (0.5 * rng.standard_normal((sets, 3 * k))).astype(np.float32)
        t = torch.from_numpy(t) if mod32 else gen.to_storage(t, dt)
        self.wide = t
        parts = {"g": t[:, :k], "c": t[:, k:2 * k], "d": t[:, 2 * k:]}
        self.at = {"g": slice(0, k), "c": slice(k, 2 * k), "d": slice(2 * k, 3 * k)}
        self.mods = {x: parts[x] for x in mods if x != "g" or branch}
        self.index = None
        if index == "any":
            self.index = torch.from_numpy(rng.integers(-1, sets + 1, m).astype(np.int32))
        elif index == "sorted":
            self.index = torch.from_numpy(np.sort(rng.integers(0, sets, m)).astype(np.int32))

    def oracle(self, eps=EPS):
        def v(t):
            return None if t is None else f32(t, self.dt)
        m = {x: v(t.contiguous()) for x, t in self.mods.items()}
        return og.rows(None if self.y is None else gen.as_numpy_bits(self.y), gen.as_numpy_bits(self.h), self.dt, self.norm,
                       v(self.w), eps, self.post, v(self.pw), self.alpha, m.get("g"), m.get("c"), m.get("d"),
                       None if self.index is None else self.index.numpy())

    def operands(self, eps=EPS):
        def d(t):
            return None if t is None else t.to(DEV)
        wide = self.wide.to(DEV)
        names = {"g": "gate", "c": "mod_scale", "d": "mod_shift"}
        return (d(self.y), d(self.h)), dict(
            weight=d(self.w), eps=eps, norm=self.norm, branch_scale=self.alpha, post=self.post, post_weight=d(self.pw),
            index=d(self.index) if self.mods else None, **{names[x]: wide[:, self.at[x]] for x in self.mods})


SHAPES = [
    dict(m=1, k=1), dict(m=3, k=7, post="layer", pw="same"), dict(m=5, k=64, norm="layer", w="same"), dict(m=2, k=513, post="rms", pw="f32", w="f32"),
    dict(m=1, k=1920, post="rms", norm="layer", mod32=True), dict(m=130, k=1920, sets=10, norm="layer", post="layer"),
    dict(m=37, k=4095, sets=37, mod32=True, post="rms"), dict(m=9, k=8192, branch=False, norm="layer"),
    dict(m=12, k=1000, sets=5, index="any", mod32=True, post="rms", pw="same"), dict(m=3, k=12289, norm="layer", mods="g"),
    dict(m=2, k=32768, post="layer", pw="f32", alpha=0.3), dict(m=2, k=32767, mods=""), dict(m=4, k=520, mods="cd", alpha=-2.0),
    dict(m=1025, k=2048, sets=25, norm="layer", post="rms", mod32=True), dict(m=1100, k=2056, sets=7, index="sorted"),
    dict(m=1024, k=4099, norm="layer", post="layer", pw="same", sets=3, index="any"), dict(m=1030, k=136, branch=False, mods="d"),
    dict(m=1026, k=16390, post="rms", norm="layer", mod32=True, sets=6), dict(m=6, k=8, norm="layer", post="layer"),
]


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("kw", SHAPES, ids=lambda k: "-".join(str(v) for v in k.values()))
def test_rows_equal_the_formula(vq, kw, dt):
    c = Case(dt=dt, **kw)
    (y, h), how = c.operands()
    n, s = vq.vq_gated_norm(y, h, **how)
    torch.cuda.synchronize()
    os_, ov = c.oracle()
    assert s is h if y is None else np.array_equal(bits(s), bits(os_))
    assert np.array_equal(bits(n), bits(onum.from_f32(ov, dt)))


@pytest.mark.parametrize("dt,nb,kw,n_out,gran", [
    ("bf16", 8, dict(m=1, k=64, post="rms"), 0, "token"),
    ("fp16", 8, dict(m=1, k=1920, norm="layer", w="f32"), 0, "token"),
    ("bf16", 8, dict(m=333, k=1920, sets=3, post="layer", pw="same", norm="layer", mod32=True), 19, "token"),
    ("bf16", 6, dict(m=70, k=1920, branch=False, sets=7), 128, "token"),
    ("fp16", 4, dict(m=5, k=64, index="any", sets=3), 1, "token"),
    ("bf16", 4, dict(m=17, k=5760, post="rms", norm="layer"), 0, "token"),
    ("fp16", 8, dict(m=9, k=12288, index="any", sets=4, w="same", post="rms", mod32=True), 64, "token"),
    ("bf16", 8, dict(m=3, k=32768, norm="layer", w="f32"), 65, "token"),
    ("bf16", 8, dict(m=19, k=1920, post="layer"), 0, "static"),
    ("fp16", 6, dict(m=6, k=4096, norm="layer", sets=6), 7, "static"),
    ("bf16", 8, dict(m=1027, k=2048, norm="layer", sets=13, post="rms", mod32=True), 0, "token"),
    ("fp16", 8, dict(m=1028, k=4160, sets=4, post="rms"), 70, "token"),
])
def test_codes_equal_the_quantizer_of_the_rows(vq, dt, nb, kw, n_out, gran):
    c = Case(dt=dt, **kw)
    k = kw["k"]
    idx = np.sort(np.random.default_rng(k).choice(k, n_out, replace=False)).astype(np.int32) if n_out else None
    st = np.array([0.03, 0.11], np.float32)[: 2 if n_out else 1] if gran == "static" else None
    (y, h), how = c.operands()
    codes, scales, s = vq.vq_gated_norm_quant(
        y, h, nb, gran=gran, idx=None if idx is None else torch.from_numpy(idx).to(DEV),
        static_scale=None if st is None else torch.from_numpy(st).to(DEV), **how)
    torch.cuda.synchronize()
    os_, ov = c.oracle()
    oc, osc = onorm.quant(ov, nb, idx, st)
    assert y is None or np.array_equal(bits(s), bits(os_))
    assert np.array_equal(bits(scales).reshape(-1), bits(osc).reshape(-1))
    assert np.array_equal(codes.cpu().numpy(), oc)


def test_width_read_on_the_device(vq):
    (y, h), how = Case(12, 640, "bf16", post="rms", norm="layer").operands()
    for nb in (4, 6, 8):
        w = torch.tensor([nb], dtype=torch.int32, device=DEV)
        a = vq.vq_gated_norm_quant(y, h, 8, bits_dev=w, **how)
        b = vq.vq_gated_norm_quant(y, h, nb, **how)
        assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("into", ["branch", "residual"])
@pytest.mark.parametrize("m,k,n_out", [(300, 4096, 0), (300, 4096, 40), (1100, 1920, 0), (40, 4093, 0), (5, 5, 0)])
def test_sum_in_place(vq, into, m, k, n_out):
    """The sum may be the residual or the branch itself, also with outlier channels gathered from both."""
    c = Case(m, k, "bf16", post="rms", norm="layer", sets=5)
    idx = torch.arange(0, k, 101, dtype=torch.int32, device=DEV)[:n_out] if n_out else None
    for quant in ([True] if n_out else [False, True] if k % 64 == 0 else [False]):
        (y, h), how = c.operands()

        def call(**kw):
            return vq.vq_gated_norm_quant(y, h, 8, idx=idx, **how, **kw) if quant else vq.vq_gated_norm(y, h, **how, **kw)
        want = call()
        t = y if into == "branch" else h
        got = call(sum_out=t)
        assert got[-1] is t and all(torch.equal(p, q) for p, q in zip(got, want))


@pytest.mark.parametrize("k,pad,shift", [(512, 8, 0), (512, 3, 0), (509, 0, 1), (512, 8, 3), (6, 1, 1)])
def test_pitches_and_addresses(vq, k, pad, shift):
    """Row slices of wider buffers, at any element address; nothing beyond a row is written."""
    m = 11
    c = Case(m, k, "bf16", post="rms", norm="layer", sets=11, w="same")
    (y, h), how = c.operands()
    want = vq.vq_gated_norm(y, h, **how)

    def wide(t=None):
        b = torch.full((m * (k + pad) + 8,), 7.0, dtype=torch.bfloat16, device=DEV)
        v = b[shift:shift + m * (k + pad)].view(m, k + pad)[:, :k]
        if t is not None:
            v.copy_(t)
        return b, v
    (_, yv), (_, hv), (nb, nv), (sb, sv) = wide(y), wide(h), wide(), wide()
    vq.vq_gated_norm(yv, hv, **how, y=nv, sum_out=sv)
    assert torch.equal(nv, want[0]) and torch.equal(sv, want[1])
    for b in (nb, sb):
        keep = torch.ones_like(b, dtype=torch.bool)
        keep[shift:shift + m * (k + pad)].view(m, k + pad)[:, :k] = False
        assert bool((b[keep] == 7.0).all())


def test_values_that_are_not_finite(vq):
    """They stay in their row; a row that uses no set keeps its residual whatever its branch holds; the
    codes' scales say NaN."""
    c = Case(8, 256, "bf16", post="rms", norm="layer", sets=3, index="sorted")
    c.index[5] = 3
    c.y[1, 7], c.y[2, 0], c.h[3, 255], c.y[5] = float("nan"), float("inf"), float("-inf"), float("nan")
    (y, h), how = c.operands()
    n, s = vq.vq_gated_norm(y, h, **how)
    codes, scales, s2 = vq.vq_gated_norm_quant(y, h, 8, **how)
    os_, ov = c.oracle()
    bad = [1, 2, 3]
    good = [i for i in range(8) if i not in bad]
    assert np.array_equal(bits(s)[good], bits(os_)[good]) and torch.equal(s[5], h[5])
    assert np.array_equal(bits(n)[good], bits(onum.from_f32(ov, "bf16"))[good])
    assert bool(n[bad].isnan().any(1).all())
    oc, osc = onorm.quant(ov[good], 8)
    assert np.array_equal(codes.cpu().numpy()[good], oc) and np.array_equal(scales.cpu().numpy()[good], osc)
    assert bool(scales[bad].isnan().all())


@pytest.mark.parametrize("where", ["gate", "mod_scale", "mod_shift", "weight", "post_weight"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("n_out", [0, 3])
def test_parameters_that_are_not_finite_show_in_the_scales(vq, where, value, n_out):
    c = Case(6, 128, "bf16", post="rms", pw="f32", w="f32", sets=2, mod32=True)
    (y, h), how = c.operands()
    idx = torch.tensor([5, 40, 99], dtype=torch.int32, device=DEV) if n_out else None
    for at in ([40] if n_out else [0, 77]):
        t = how[where].clone()
        t[..., at] = value
        _, scales, _ = vq.vq_gated_norm_quant(y, h, 8, idx=idx, **{**how, where: t})
        assert bool(scales.isnan().all())


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_large_means_and_constant_rows(vq, dt):
    c = Case(4, 640, dt, branch=False, norm="layer", mods="")
    big = 4000.0 if dt == "fp16" else 250.0
    rng = np.random.default_rng(8)
    c.h = gen.to_storage((big + rng.integers(-2, 3, (4, 640)) * (4.0 if dt == "fp16" else 1.0)).astype(np.float32), dt)
    c.h[1] = big
    c.h[2] = 0.0
    (_, h), how = c.operands()
    n, _ = vq.vq_gated_norm(None, h, **how)
    _, ov = c.oracle()
    assert np.array_equal(bits(n), bits(onum.from_f32(ov, dt)))
    assert not n[1:3].any()


def test_no_rows_and_the_whole_range_of_a_type(vq):
    h = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV)
    n, s = vq.vq_gated_norm(h, h, gate=torch.ones(3, 64, device=DEV))
    assert n.shape == s.shape == (0, 64)
    big = torch.full((2, 64), 3e38, dtype=torch.bfloat16, device=DEV)
    big[:, ::2] *= -1
    n, _ = vq.vq_gated_norm(None, big, norm="layer")
    assert bool((n.abs() == 1).all())
    tiny = torch.full((1, 64), 1e-38, dtype=torch.bfloat16, device=DEV)
    n, _ = vq.vq_gated_norm(None, tiny, eps=0.0)
    assert bool((n == 1).all())


def test_other_stream_and_replayed_graph(vq):
    c = Case(50, 1920, "bf16", post="rms", norm="layer", sets=5, index="any", mod32=True)
    (y, h), how = c.operands()
    n, s = torch.empty_like(h), torch.empty_like(h)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        vq.vq_gated_norm(y, h, **how, y=n, sum_out=s)
        side.synchronize()
        want = (n.clone(), s.clone())
        with torch.cuda.graph(graph, stream=side):
            vq.vq_gated_norm(y, h, **how, y=n, sum_out=s)
    torch.cuda.synchronize()
    for i in range(3):
        if i:
            y.copy_(torch.randn_like(y))
            how["index"].copy_(torch.randint(-1, 6, (50,), device=DEV))
            want = vq.vq_gated_norm(y, h, **how)
        n.zero_(), s.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(n, want[0]) and torch.equal(s, want[1])
