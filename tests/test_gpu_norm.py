"""GPU parity of the root-mean-square norm with the residual's addition, as 16-bit rows and
as activation codes (oracle/norm.py).

The sum of squares is float64 on both sides and every later step is one float32 operation
or one rounding, so outputs, codes and scales must equal the oracle's bit for bit.
"""
import numpy as np
import pytest
import torch

import gen
from oracle import norm as onorm
from oracle import numerics as onum

pytestmark = pytest.mark.gpu

DEV = "cuda"
TD = {"bf16": torch.bfloat16, "fp16": torch.float16}
EPS = 1e-6


@pytest.fixture(scope="module")
def vq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_quantized_linear_vq_amd as m
    return m


def npb(t):
    return gen.as_numpy_bits(t.cpu().contiguous())


def bits(a):
    a = np.ascontiguousarray(a)
    return a.view(np.uint16 if a.dtype.itemsize == 2 else np.uint32 if a.dtype.itemsize == 4 else a.dtype)


def make(m, k, dt, res, w, seed=0):
    rng = np.random.default_rng([m, k, seed])
    x = rng.standard_normal((m, k)).astype(np.float32)
    x[:, :: max(1, k // 5)] *= 20.0
    xs = gen.to_storage(x, dt)
    rs = gen.to_storage((2 * rng.standard_normal((m, k))).astype(np.float32), dt) if res else None
    wv = (1 + 0.2 * rng.standard_normal(k)).astype(np.float32)
    ws = None if w == "none" else torch.from_numpy(wv) if w == "f32" else gen.to_storage(wv, dt)
    wf = None if w == "none" else wv if w == "f32" else onum.to_f32(gen.as_numpy_bits(ws), dt)
    return xs, rs, ws, wf


def dev(t):
    return None if t is None else t.to(DEV)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("m,k,res,w", [
    (1, 1, False, "same"), (3, 7, True, "same"), (5, 64, False, "none"), (2, 513, True, "f32"),
    (1, 1920, True, "same"), (130, 1920, True, "f32"), (37, 4095, True, "same"), (9, 8192, False, "f32"),
    (3, 12289, True, "same"), (2, 32768, True, "same"), (2, 32767, False, "none"), (4, 520, True, "none"),
])
def test_rows_equal_the_formula(vq, m, k, res, w, dt):
    x, r, ws, wf = make(m, k, dt, res, w)
    got = vq.vq_rmsnorm(dev(x), dev(ws), EPS, residual=dev(r))
    torch.cuda.synchronize()
    h, v = onorm.rows(gen.as_numpy_bits(x), dt, wf, EPS, None if r is None else gen.as_numpy_bits(r))
    y = got[0] if res else got
    if res:
        assert np.array_equal(bits(npb(got[1])), bits(h))
    assert np.array_equal(bits(npb(y)), bits(onum.from_f32(v, dt)))


@pytest.mark.parametrize("m,k,dt,nb,res,w,n_out,gran", [
    (1, 64, "bf16", 8, True, "same", 0, "token"),
    (1, 1920, "fp16", 8, True, "f32", 0, "token"),
    (333, 1920, "bf16", 8, True, "same", 19, "token"),
    (70, 1920, "bf16", 6, False, "none", 128, "token"),
    (5, 64, "fp16", 4, True, "same", 1, "token"),
    (17, 5760, "bf16", 4, True, "same", 0, "token"),
    (9, 12288, "fp16", 8, True, "same", 64, "token"),
    (3, 32768, "bf16", 8, False, "f32", 65, "token"),
    (19, 1920, "bf16", 8, True, "same", 0, "static"),
    (6, 4096, "fp16", 6, True, "same", 7, "static"),
])
def test_codes_equal_the_quantizer_of_the_normed_rows(vq, m, k, dt, nb, res, w, n_out, gran):
    x, r, ws, wf = make(m, k, dt, res, w, nb)
    idx = None
    if n_out:
        idx = torch.from_numpy(np.sort(np.random.default_rng(k).choice(k, n_out, replace=False)).astype(np.int32))
    st = torch.tensor([0.03, 0.11][: 2 if n_out else 1]) if gran == "static" else None
    got = vq.vq_rmsnorm_quant(dev(x), dev(ws), nb, EPS, residual=dev(r), gran=gran, idx=dev(idx), static_scale=dev(st))
    torch.cuda.synchronize()
    h, v = onorm.rows(gen.as_numpy_bits(x), dt, wf, EPS, None if r is None else gen.as_numpy_bits(r))
    codes, scales = onorm.quant(v, nb, None if idx is None else idx.numpy(), None if st is None else st.numpy())
    assert np.array_equal(got[1].cpu().numpy().reshape(-1).view(np.uint32), scales.reshape(-1).view(np.uint32))
    assert np.array_equal(got[0].cpu().numpy(), codes)
    if res:
        assert np.array_equal(bits(npb(got[2])), bits(h))


def test_width_read_on_the_device(vq):
    x, r, ws, _ = make(12, 640, "bf16", True, "same")
    for nb in (4, 6, 8):
        w = torch.tensor([nb], dtype=torch.int32, device=DEV)
        a = vq.vq_rmsnorm_quant(dev(x), dev(ws), 8, EPS, residual=dev(r), bits_dev=w)
        b = vq.vq_rmsnorm_quant(dev(x), dev(ws), nb, EPS, residual=dev(r))
        assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("into", ["x", "residual"])
@pytest.mark.parametrize("n_out", [0, 40])
def test_sum_in_place(vq, into, n_out):
    """h may be x or the residual itself, also with outlier channels gathered from both."""
    x, r, ws, _ = make(300, 4096, "bf16", True, "same")
    idx = torch.arange(0, 4096, 101, dtype=torch.int32, device=DEV)[:n_out] if n_out else None
    want = vq.vq_rmsnorm_quant(dev(x), dev(ws), 8, EPS, residual=dev(r), idx=idx)
    xd, rd = dev(x), dev(r)
    t = xd if into == "x" else rd
    got = vq.vq_rmsnorm_quant(xd, dev(ws), 8, EPS, residual=rd, idx=idx, sum_out=t)
    assert got[2] is t and all(torch.equal(p, q) for p, q in zip(got, want))
    xd, rd = dev(x), dev(r)
    t = xd if into == "x" else rd
    got = vq.vq_rmsnorm(xd, dev(ws), EPS, residual=rd, sum_out=t)
    want = vq.vq_rmsnorm(dev(x), dev(ws), EPS, residual=dev(r))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("k,pad,shift", [(512, 8, 0), (512, 3, 0), (509, 0, 1), (512, 8, 3)])
def test_pitches_and_addresses(vq, k, pad, shift):
    """Row slices of wider buffers, at any element address; nothing beyond a row is written."""
    m = 11
    x, r, ws, _ = make(m, k, "bf16", True, "same")
    want = vq.vq_rmsnorm(dev(x), dev(ws), EPS, residual=dev(r))

    def wide(t=None):
        b = torch.full((m * (k + pad) + 8,), 7.0, dtype=torch.bfloat16, device=DEV)
        v = b[shift:shift + m * (k + pad)].view(m, k + pad)[:, :k]
        if t is not None:
            v.copy_(t)
        return b, v
    (_, xv), (_, rv), (yb, yv), (hb, hv) = wide(x), wide(r), wide(), wide()
    vq.vq_rmsnorm(xv, dev(ws), EPS, residual=rv, y=yv, sum_out=hv)
    assert torch.equal(yv, want[0]) and torch.equal(hv, want[1])
    for b, v in ((yb, yv), (hb, hv)):
        v.fill_(7.0)
        assert bool((b == 7.0).all())


def test_rows_with_infinities_and_nan(vq):
    """A row with an infinity or NaN gets a NaN scale; the other rows are as without it."""
    x, _, ws, _ = make(8, 640, "fp16", False, "same")
    clean = vq.vq_rmsnorm_quant(dev(x), dev(ws), 8, EPS)
    bad = x.clone()
    bad[2, 5] = float("inf")
    bad[4, 639] = float("-inf")
    bad[7, 0] = float("nan")
    c, s = vq.vq_rmsnorm_quant(dev(bad), dev(ws), 8, EPS)
    rows = torch.tensor([2, 4, 7], device=DEV)
    keep = torch.tensor([0, 1, 3, 5, 6], device=DEV)
    assert bool(torch.isnan(s[rows]).all())
    assert torch.equal(s[keep], clean[1][keep]) and torch.equal(c[keep], clean[0][keep])
    y = vq.vq_rmsnorm(dev(bad), dev(ws), EPS)
    assert bool(torch.isnan(y[rows]).any(1).all()) and bool(torch.isfinite(y[keep].float()).all())


def test_rows_of_zeros(vq):
    x = torch.zeros((3, 128), dtype=torch.bfloat16, device=DEV)
    c, s = vq.vq_rmsnorm_quant(x, None, 8, EPS)
    assert not c.any() and not s.any()
    assert not vq.vq_rmsnorm(x, None, EPS).any()


def test_no_rows(vq):
    x = torch.empty((0, 128), dtype=torch.bfloat16, device=DEV)
    assert vq.vq_rmsnorm(x, None).shape == (0, 128)
    c, s, h = vq.vq_rmsnorm_quant(x, None, 8, residual=x)
    assert c.shape == (0, 128) and s.shape == (0,) and h.shape == (0, 128)


def test_captured_and_replayed_on_a_side_stream(vq):
    x, r, ws, _ = make(200, 1920, "bf16", True, "same")
    x2, r2, _, _ = make(200, 1920, "bf16", True, "same", 9)
    xb, rb, wd = dev(x), dev(r), dev(ws)
    codes = torch.empty((200, 1920), dtype=torch.int8, device=DEV)
    scales = torch.empty(200, device=DEV)
    h = torch.empty_like(xb)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            vq.vq_rmsnorm_quant(xb, wd, 8, EPS, residual=rb, codes=codes, scales=scales, sum_out=h)
    torch.cuda.synchronize()
    for a, b in ((x, r), (x2, r2), (x, r2)):
        xb.copy_(a)
        rb.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        want = vq.vq_rmsnorm_quant(dev(a), wd, 8, EPS, residual=dev(b))
        assert torch.equal(codes, want[0]) and torch.equal(scales, want[1]) and torch.equal(h, want[2])


def test_refusals(vq):
    x = torch.zeros((4, 128), dtype=torch.bfloat16, device=DEV)
    w = torch.ones(128, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(TypeError):
        vq.vq_rmsnorm(x.float(), w)
    with pytest.raises(TypeError):
        vq.vq_rmsnorm(x, w.half())
    with pytest.raises(TypeError):
        vq.vq_rmsnorm(x.cpu(), w)
    with pytest.raises(ValueError):
        vq.vq_rmsnorm(x, w[:64])
    with pytest.raises(ValueError):
        vq.vq_rmsnorm(x, w, residual=x[:2])
    with pytest.raises(ValueError):
        vq.vq_rmsnorm(x, w, sum_out=x)
    with pytest.raises(ValueError):
        vq.vq_rmsnorm(x.t(), w)
    with pytest.raises(ValueError):
        vq.vq_rmsnorm(x[:1].expand(4, 128), w)
    for kw in (dict(eps=-1.0), dict(eps=float("nan"))):
        with pytest.raises(vq.VQError):
            vq.vq_rmsnorm(x, w, **kw)
    for kw in (dict(bits=5), dict(bits=8, gran="tensor"), dict(bits=8, gran="row"), dict(bits=8, gran="static")):
        with pytest.raises(vq.VQError):
            vq.vq_rmsnorm_quant(x, w, **kw)
    with pytest.raises(vq.VQError):
        vq.vq_rmsnorm_quant(x[:, :100], None, 8)  # K % 64
    with pytest.raises(vq.VQError):
        vq.vq_rmsnorm(torch.zeros((1, 32769), dtype=torch.bfloat16, device=DEV), None)


@pytest.mark.parametrize("m,k", [(1100, 64), (1030, 4088), (1500, 2056), (1024, 12288), (1200, 9), (1025, 15), (2000, 3)])
def test_many_rows(vq, m, k):
    """Row counts that take several pieces a thread, every way a row can end."""
    x, r, ws, wf = make(m, k, "bf16", True, "f32", 5)
    y, hs = vq.vq_rmsnorm(dev(x), dev(ws), EPS, residual=dev(r))
    torch.cuda.synchronize()
    h, v = onorm.rows(gen.as_numpy_bits(x), "bf16", wf, EPS, gen.as_numpy_bits(r))
    assert np.array_equal(bits(npb(hs)), bits(h)) and np.array_equal(bits(npb(y)), bits(onum.from_f32(v, "bf16")))
    xd = dev(x)  # in place, rows that end in an overlapping piece too
    y2, h2 = vq.vq_rmsnorm(xd, dev(ws), EPS, residual=dev(r), sum_out=xd)
    assert torch.equal(y2, y) and torch.equal(h2, hs)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_weights_that_are_not_finite(vq, bad):
    x, _, ws, _ = make(5, 640, "bf16", False, "same")
    ws = ws.clone()
    ws[77] = bad
    _, s = vq.vq_rmsnorm_quant(dev(x), dev(ws), 8, EPS)
    assert bool(torch.isnan(s).all())


def test_codes_of_a_norm_equal_those_of_its_rows_when_exact(vq):
    """Rows whose normed values are 16-bit already: the fused codes equal the quantizer's."""
    x = torch.zeros((4, 256), dtype=torch.bfloat16, device=DEV)
    x[:, :64] = 2.0
    x[1, :64] = -4.0  # every row's mean square is a power of four: rstd exact
    c, s = vq.vq_rmsnorm_quant(x, None, 8, 0.0)
    y = vq.vq_rmsnorm(x, None, 0.0)
    c2, s2 = vq.vq_quant_act(y, 8, "token")
    assert torch.equal(c, c2) and torch.equal(s, s2)


@pytest.mark.parametrize("m,k", [(17776, 1920), (6500, 4095), (3700, 9001)])
@pytest.mark.parametrize("res", [False, True])
def test_larger_than_the_cache(vq, m, k, res):
    """Rows do not depend on one another: the whole call, the sum in place of the residual, gives
    bit for bit what calls of few rows give (which the oracle pins above)."""
    if not res:
        m *= 2
    g = torch.Generator(device=DEV).manual_seed(m + k)
    x = torch.randn(m, k, device=DEV, generator=g).bfloat16()
    r = torch.randn(m, k, device=DEV, generator=g).bfloat16() if res else None
    w = torch.randn(k, device=DEV, generator=g).bfloat16()
    h = r.clone() if res else None
    got = vq.vq_rmsnorm(x, w, EPS, residual=h, sum_out=h)
    y = got[0] if res else got
    if k % 64 == 0:
        h2 = r.clone() if res else None
        codes, scales = vq.vq_rmsnorm_quant(x, w, 8, EPS, residual=h2, sum_out=h2)[:2]
    for i in range(0, m, 900):
        s = slice(i, min(m, i + 900))
        part = vq.vq_rmsnorm(x[s], w, EPS, residual=r[s] if res else None)
        if res:
            assert torch.equal(h[s], part[1])
        assert torch.equal(y[s], part[0] if res else part)
        if k % 64 == 0:
            part = vq.vq_rmsnorm_quant(x[s], w, 8, EPS, residual=r[s] if res else None)
            assert torch.equal(codes[s], part[0]) and torch.equal(scales[s], part[1])
            if res:
                assert torch.equal(h2[s], part[2])
