"""GPU parity of the experts' products (oracle/experts.py): the integer form bit for bit
against the oracle's exact accumulators and epilogue, the 16-bit form within the float32
summation bound of the unquantized layer."""
import numpy as np
import pytest
import torch

import gen
from oracle import dense, experts
from oracle import numerics as onum
from oracle import quantizer

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


def i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device=DEV)


def offsets_of(counts, first=0):
    return np.concatenate([[first], first + np.cumsum(counts)]).astype(np.int32)


def operands(m, e, n, k, bits, seed):
    rng = np.random.default_rng([m, e, n, k, seed])
    a = np.clip(np.rint(rng.standard_normal((m, k)) * 40), -127, 127).astype(np.int8)
    sa = (0.01 + 0.02 * rng.random(m)).astype(np.float32)
    q = 127 if bits == 8 else 7
    b = np.clip(np.rint(rng.standard_normal((e * n, k)) * q / 3), -q, q).astype(np.int8)
    sb = (0.001 + 0.001 * rng.random(e * n)).astype(np.float32)
    return a, sa, b, sb


def pieces(b):
    rows, rb = b.shape
    p = (rb + 63) // 64
    f = np.zeros((rows, p * 64), dtype=b.dtype)
    f[:, :rb] = b
    return np.ascontiguousarray(f.reshape(rows, p, 64).transpose(1, 0, 2))


def int_reference(a, sa, b, sb, n, off, rows, t, out):
    """Bit patterns of the outputs, and which rows are written."""
    y = np.zeros((t, n), dtype=np.float32)
    own = np.zeros(t, dtype=bool)
    for e in range(len(off) - 1):
        lo, hi = off[e], off[e + 1]
        if hi <= lo:
            continue
        own[lo:hi] = True
        idx = np.arange(lo, hi) if rows is None else rows[lo:hi]
        ok = (idx >= 0) & (idx < len(a))
        i = idx[ok]
        be = b[e * n:(e + 1) * n]
        acc = a[i].astype(np.float64) @ be.astype(np.float64).T  # exact: below 2^53
        scale = (sa[i][:, None] * sb[None, e * n:(e + 1) * n]).astype(np.float32)
        part = np.zeros((hi - lo, n), dtype=np.float32)
        part[ok] = (acc.astype(np.float32) * scale).astype(np.float32)
        y[lo:hi] = part
    return onum.from_f32(y, out), own


def check_int(vq, a, sa, b, sb, n, off, rows, t, bits, out, kblock, y=None):
    packed = b if bits == 8 else quantizer.pack_int4(b)
    bd = torch.from_numpy(pieces(packed) if kblock else packed).to(DEV)
    if y is None:
        y = torch.full((t, n), 7.0, dtype=TD[out], device=DEV)
    vq.vq_qgemm_experts(torch.from_numpy(a).to(DEV), torch.from_numpy(sa).to(DEV), bd, torch.from_numpy(sb).to(DEV),
                        bits, i32(off), rows=None if rows is None else i32(rows), y=y)
    torch.cuda.synchronize()
    want, own = int_reference(a, sa, b, sb, n, off, rows, t, out)
    got = npb(y)
    view = np.uint32 if out == "fp32" else np.uint16
    g, w = got[own].view(view), np.ascontiguousarray(want[own]).view(view)
    # a zero has either sign where an index outside a zeroes the row
    assert np.array_equal(np.where(onum.to_f32(got[own], out) == 0, 0, g), np.where(onum.to_f32(want[own], out) == 0, 0, w))
    assert bool((y[torch.from_numpy(~own).to(DEV)] == 7.0).all())


INT_CASES = [
    # counts per expert, n, k, bits, pieces, gathered, out
    ([1], 1, 64, 8, False, False, "fp32"),
    ([1], 33, 64, 4, True, False, "bf16"),
    ([0, 1, 0, 2], 100, 192, 8, True, True, "fp16"),
    ([2] * 16, 260, 512, 4, True, True, "bf16"),
    ([3, 0, 0, 40, 1, 0], 64, 1920, 8, False, True, "bf16"),
    ([5, 33, 31, 32, 64, 65], 257, 320, 4, False, False, "fp32"),
    ([300, 0, 513], 300, 448, 8, True, False, "bf16"),
    ([256, 256], 256, 256, 8, False, False, "fp16"),
    ([1000, 3, 700], 520, 640, 4, True, True, "bf16"),
    ([129, 127, 128, 1], 255, 1088, 8, True, True, "fp32"),
    ([700, 900, 1100, 20], 1030, 192, 8, False, True, "bf16"),
    ([0, 0, 600, 0], 1030, 576, 4, False, False, "bf16"),
    ([1] * 130, 40, 64, 8, False, True, "bf16"),
    ([7] * 70, 65, 128, 4, True, False, "fp16"),
    ([0, 0, 0], 16, 64, 8, False, False, "bf16"),
]


@pytest.mark.parametrize("counts,n,k,bits,kblock,gather,out", INT_CASES)
def test_codes_product_equals_the_layer_bit_for_bit(vq, counts, n, k, bits, kblock, gather, out):
    off = offsets_of(counts)
    t = int(off[-1])
    if t == 0:
        t = 3  # rows that no expert owns
    m = max(1, t // 2) if gather else t
    a, sa, b, sb = operands(m, len(counts), n, k, bits, 1)
    rows = np.random.default_rng(t).integers(0, m, t).astype(np.int32) if gather else None
    check_int(vq, a, sa, b, sb, n, off, rows, t, bits, out, kblock)


@pytest.mark.parametrize("bits,scale", [(8, 20), (4, 20), (8, 600)])
def test_rows_outside_the_offsets_and_bad_indices(vq, bits, scale):
    """Rows before the first and behind the last offset keep what they held; an index outside
    the codes gives a row of zeros."""
    off = offsets_of([scale, 0, scale + 13], first=5)
    t = int(off[-1]) + 9
    a, sa, b, sb = operands(scale, 3, 96, 128, bits, 2)
    rows = np.random.default_rng(3).integers(0, scale, t).astype(np.int32)
    rows[7], rows[int(off[1]) + 1], rows[int(off[-1]) - 1] = -1, scale, 2 ** 31 - 1
    check_int(vq, a, sa, b, sb, 96, off, rows, t, bits, "bf16", False)


def test_offsets_out_of_range_stay_inside_the_buffers(vq):
    """Offsets below zero or beyond the rows are clamped: rows that a valid prefix owns are
    right, and nothing outside y is written."""
    a, sa, b, sb = operands(40, 2, 64, 64, 8, 3)
    buf = torch.full((60, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    off = i32([-50, 20, 10 ** 9])
    vq.vq_qgemm_experts(torch.from_numpy(a).to(DEV), torch.from_numpy(sa).to(DEV), torch.from_numpy(b).to(DEV),
                        torch.from_numpy(sb).to(DEV), 8, off, y=buf[10:50])
    torch.cuda.synchronize()
    want, _ = int_reference(a, sa, b, sb, 64, np.array([0, 20, 40]), None, 40, "bf16")
    assert np.array_equal(npb(buf[10:50]), want)
    assert bool((buf[:10] == 7.0).all()) and bool((buf[50:] == 7.0).all())


def test_one_expert_equals_the_layer(vq):
    x = gen.make_x(2, m=700).to(DEV)
    w = gen.make_w(2, n=640).to(DEV)
    for bits in (8, 4):
        for kb in (False, True):
            wc, ws = vq.vq_pack_weights(w, bits, kblock=kb)
            ac, sa = vq.vq_quant_act(x, 8, "token")
            got = vq.vq_qgemm_experts(ac, sa, wc, ws, bits, i32([0, 700]))
            assert torch.equal(got, vq.vq_qgemm_dequant(ac, sa, wc, ws, bits))


def test_pitched_output(vq):
    a, sa, b, sb = operands(50, 2, 70, 128, 8, 4)
    big = torch.full((50, 75), 7.0, dtype=torch.bfloat16, device=DEV)
    check_int(vq, a, sa, b, sb, 70, offsets_of([20, 30]), None, 50, 8, "bf16", False, y=big[:, :70])
    assert bool((big[:, 70:] == 7.0).all())


def half_step(ex, b, out):
    if out == "fp32":
        return b
    mant, emin = (7, -126) if out == "bf16" else (10, -14)
    return b + 0.5 * np.exp2(np.floor(np.log2(np.maximum(np.abs(ex) + b, 2.0 ** emin))) - mant)


@pytest.mark.parametrize("counts,n,k,dt,out,gather", [
    ([1], 1, 64, "bf16", "bf16", False),
    ([0, 2, 1], 70, 128, "fp16", "fp32", True),
    ([2] * 12, 260, 512, "bf16", "bf16", True),
    ([40, 0, 33, 1], 100, 1920, "fp16", "fp16", True),
    ([300, 0, 520], 300, 192, "bf16", "fp32", False),
    ([257, 255, 700], 515, 256, "fp16", "bf16", True),
    ([900, 100], 1030, 64, "bf16", "bf16", False),
])
def test_dense_product_within_the_float32_bound(vq, counts, n, k, dt, out, gather):
    rng = np.random.default_rng([n, k])
    off = offsets_of(counts)
    t = int(off[-1])
    m = max(1, t // 2) if gather else t
    x = gen.to_storage(rng.standard_normal((m, k)).astype(np.float32), dt)
    w = gen.to_storage((rng.standard_normal((len(counts) * n, k)) * 0.02).astype(np.float32), dt).reshape(len(counts), n, k)
    rows = rng.integers(0, m, t).astype(np.int32) if gather else None
    y = vq.vq_gemm_dense_experts(x.to(DEV), w.to(DEV), i32(off), rows=None if rows is None else i32(rows), out_dtype=TD[out])
    torch.cuda.synchronize()
    xs, ws = npb(x), npb(w)
    ex = experts.apply(off, rows, t, n, lambda e, i: dense.exact(xs[i], dt, ws[e]))
    mag = experts.apply(off, rows, t, n, lambda e, i: dense.magnitude(xs[i], dt, ws[e]))
    err = np.abs(y.float().cpu().numpy().astype(np.float64) - ex)
    b = half_step(ex, dense.bound(mag, k), out)
    assert np.all(err <= b + 1e-300), float((err / np.maximum(b, 1e-300)).max())


def test_dense_pitches_and_expert_strides(vq):
    rng = np.random.default_rng(12)
    e, n, k, m = 3, 50, 128, 90
    wide = gen.to_storage((rng.standard_normal((e * (n + 4), k + 24)) * 0.02).astype(np.float32), "bf16").to(DEV)
    w = wide.view(e, n + 4, k + 24)[:, :n, :k]
    x = gen.to_storage(rng.standard_normal((m, k + 8)).astype(np.float32), "bf16").to(DEV)[:, :k]
    off = i32(offsets_of([30, 25, 35]))
    got = vq.vq_gemm_dense_experts(x, w, off)
    assert torch.equal(got, vq.vq_gemm_dense_experts(x.contiguous(), w.contiguous(), off))
    shared = vq.vq_gemm_dense_experts(x, w[:1].expand(e, n, k), off)  # every expert the same weights
    assert torch.equal(shared, vq.vq_gemm_dense_experts(x, w[:1].contiguous().expand(e, n, k).contiguous(), off))


def test_replayed_with_other_offsets(vq):
    """The launch depends on sizes alone: a captured call follows the offsets and rows that
    the buffers hold at the replay."""
    for t, n, k, e in ((24, 320, 256, 6), (900, 300, 192, 3)):
        a, sa, b, sb = operands(t, e, n, k, 8, 6)
        ad, sad, bd, sbd = (torch.from_numpy(v).to(DEV) for v in (a, sa, b, sb))
        off, rows = i32(np.zeros(e + 1)), i32(np.arange(t))
        y = torch.full((t, n), 7.0, dtype=torch.bfloat16, device=DEV)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side):
            with torch.cuda.graph(graph, stream=side):
                vq.vq_qgemm_experts(ad, sad, bd, sbd, 8, off, rows=rows, y=y)
        torch.cuda.synchronize()
        rng = np.random.default_rng(t)
        for _ in range(4):
            cut = np.sort(rng.integers(0, t + 1, e - 1))
            o = np.concatenate([[0], cut, [t]]).astype(np.int32)
            r = rng.permutation(t).astype(np.int32)
            off.copy_(torch.from_numpy(o))
            rows.copy_(torch.from_numpy(r))
            graph.replay()
            torch.cuda.synchronize()
            want, _ = int_reference(a, sa, b, sb, n, o, r, t, "bf16")
            assert np.array_equal(npb(y), want)


def test_two_streams_at_once(vq):
    cases = []
    for i in range(2):
        a, sa, b, sb = operands(600, 4, 520, 640, 8, 20 + i)
        off = offsets_of([100, 250, 0, 250])
        cases.append((a, sa, b, sb, off))
    dev_args = [[torch.from_numpy(v).to(DEV) for v in c[:4]] + [i32(c[4])] for c in cases]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    ys = []
    for _ in range(3):
        ys = []
        for st, d in zip(streams, dev_args):
            with torch.cuda.stream(st):
                ys.append(vq.vq_qgemm_experts(*d[:4], 8, d[4]))
    torch.cuda.synchronize()
    for c, y in zip(cases, ys):
        want, _ = int_reference(*c[:4], 520, c[4], None, 600, "bf16")
        assert np.array_equal(npb(y), want)


def test_no_rows_and_refusals(vq):
    a, sa, b, sb = (torch.from_numpy(v).to(DEV) for v in operands(4, 2, 32, 64, 8, 7))
    off = i32([0, 2, 4])
    assert vq.vq_qgemm_experts(a[:0], sa[:0], b, sb, 8, i32([0, 0, 0])).shape == (0, 32)
    assert vq.vq_qgemm_experts(a, sa, b, sb, 8, i32([0, 0, 0]), rows=i32([])).shape == (0, 32)
    with pytest.raises(TypeError):
        vq.vq_qgemm_experts(a, sa, b, sb, 8, off.long())
    with pytest.raises(TypeError):
        vq.vq_qgemm_experts(a, sa, b, sb, 4, off)
    with pytest.raises(ValueError):
        vq.vq_qgemm_experts(a, sa, b, sb, 8, i32([0, 1, 2, 4]))  # 64 rows over three experts
    with pytest.raises(ValueError):
        vq.vq_qgemm_experts(a, sa[:3], b, sb, 8, off)
    with pytest.raises(TypeError):
        vq.vq_qgemm_experts(a, sa, b, sb, 8, off.cpu())
    with pytest.raises(vq.VQError):
        vq.vq_qgemm_experts(a, sa, b, sb, 6, off)
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device=DEV)
    w = torch.zeros((2, 32, 64), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError):
        vq.vq_gemm_dense_experts(x, w, i32([0, 4]))
    with pytest.raises(TypeError):
        vq.vq_gemm_dense_experts(x, w.half(), off)
    with pytest.raises(ValueError):
        vq.vq_gemm_dense_experts(x, w.transpose(1, 2), off)
    with pytest.raises(vq.VQError):
        vq.vq_gemm_dense_experts(x[:, :32], w[:, :, :32], off)  # K % 64


@pytest.mark.parametrize("counts,n,k,bits", [
    ([1] * 1000, 24, 64, 8),                        # many experts, a row each
    ([0] * 500 + [600] + [0] * 499 + [70], 300, 128, 4),  # two of a thousand, in another order of tables
    ([64, 65, 128, 129, 1, 255, 257, 0, 300], 700, 192, 8),  # tails of every height
    ([20] * 30, 512, 448, 4),
    ([100], 2048, 256, 8),                          # one short tile a column, cut by columns
    ([250, 3], 1030, 320, 4),
    ([4196], 4096, 128, 8),                         # whole rounds of 256 tiles, then a tail cut by columns
    ([4096 + 70, 20], 4096, 192, 4),
    ([4096 + 200], 4096, 64, 8),                    # and one cut by rows
])
def test_tables_and_pieces(vq, counts, n, k, bits):
    off = offsets_of(counts)
    t = int(off[-1])
    a, sa, b, sb = operands(t, len(counts), n, k, bits, 31)
    check_int(vq, a, sa, b, sb, n, off, None, t, bits, "bf16", True)


@pytest.mark.parametrize("t", [30, 900])
def test_dense_rows_of_zeros_for_bad_indices(vq, t):
    """An index outside x gives zeros even where x's first row is not finite."""
    rng = np.random.default_rng(t)
    x = gen.to_storage(rng.standard_normal((t, 128)).astype(np.float32), "bf16").to(DEV)
    x[0] = float("nan")
    x[1] = float("inf")
    w = gen.to_storage((rng.standard_normal((2 * 70, 128)) * 0.1).astype(np.float32), "bf16").to(DEV).view(2, 70, 128)
    rows = torch.arange(t, dtype=torch.int32, device=DEV)
    rows[3], rows[t // 2], rows[t - 1] = -5, t, 2 ** 31 - 1
    off = i32([0, t // 3, t])
    y = vq.vq_gemm_dense_experts(x, w, off, rows=rows)
    bad = torch.tensor([3, t // 2, t - 1], device=DEV)
    assert not y[bad].any()
    keep = torch.ones(t, dtype=torch.bool, device=DEV)
    keep[bad] = False
    keep[:2] = False
    want = vq.vq_gemm_dense_experts(x, w, off)
    assert torch.equal(y[keep], want[keep]) and bool(torch.isnan(y[0]).all())


def test_offsets_that_do_not_ascend(vq):
    """Unspecified rows, but nothing outside y."""
    for t, off in ((40, [0, 30, 10, 40]), (900, [0, 800, 100, 900]), (900, [900, 0, 900, 0])):
        a, sa, b, sb = operands(t, 3, 64, 64, 8, 41)
        buf = torch.full((t + 20, 64), 7.0, dtype=torch.bfloat16, device=DEV)
        vq.vq_qgemm_experts(torch.from_numpy(a).to(DEV), torch.from_numpy(sa).to(DEV), torch.from_numpy(b).to(DEV),
                            torch.from_numpy(sb).to(DEV), 8, i32(off), y=buf[10:t + 10])
        torch.cuda.synchronize()
        assert bool((buf[:10] == 7.0).all()) and bool((buf[t + 10:] == 7.0).all())


@pytest.mark.parametrize("counts,n,k,bits,pad,shift,out", [
    ([300, 0, 513], 255, 128, 8, 0, 0, "bf16"), ([300, 0, 513], 256, 128, 8, 0, 1, "fp16"),
    ([300, 0, 513], 256, 64, 4, 1, 0, "bf16"), ([300, 65, 513], 257, 64, 8, 0, 1, "bf16"),
    ([300, 33, 513], 263, 64, 8, 2, 0, "fp16"), ([300, 1, 513], 264, 64, 8, 3, 1, "bf16"),
    ([700, 127, 1], 321, 192, 4, 0, 0, "bf16"), ([700, 128, 3], 327, 64, 8, 4, 1, "bf16"),
    ([700, 129, 3], 335, 64, 8, 0, 0, "fp16"), ([700, 200, 3], 65, 64, 8, 0, 1, "bf16"),
    ([4000, 3990, 4100, 3901], 2049, 64, 8, 0, 0, "bf16"), ([4000, 3990, 4100, 3901], 2048, 192, 4, 1, 1, "bf16"),
    ([60] * 8, 8191, 192, 8, 0, 0, "bf16"),
])
def test_rows_that_start_at_odd_elements(vq, counts, n, k, bits, pad, shift, out):
    """Every output is written, and nothing before, between or behind the rows."""
    off = offsets_of(counts)
    t = int(off[-1])
    a, sa, b, sb = operands(t, len(counts), n, k, bits, 3)
    buf = torch.full((t * (n + pad) + shift + 8,), 7.0, dtype=TD[out], device=DEV)
    y = buf[shift:shift + t * (n + pad)].view(t, n + pad)
    check_int(vq, a, sa, b, sb, n, off, None, t, bits, out, True, y=y[:, :n])
    assert bool((y[:, n:] == 7.0).all()) and bool((buf[:shift] == 7.0).all())
    assert bool((buf[shift + t * (n + pad):] == 7.0).all())
