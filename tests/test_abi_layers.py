"""C-ABI checks, without a GPU, of the norm, the group-scaled 4-bit weights and the experts'
products: invalid arguments get the documented status before any HIP call, and calls with
no rows return without one."""
import ctypes
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "bit_quantized_linear_vq_amd", "libvq.so")

# The calls pass a fake device address to entry points that must reject them: only where no
# GPU could be reached by one that does not.
pytestmark = [
    pytest.mark.skipif(not os.path.exists(LIB), reason="libvq.so not built"),
    pytest.mark.skipif(os.path.exists("/dev/kfd"), reason="a GPU is present: fake device addresses must not reach it"),
]

OK, INVALID, SHAPE, UNSUP, HIP = range(5)
F16, BF16, F32 = 0, 1, 2
FAKE = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10008)
NULL = None
NAN = float("nan")


@pytest.fixture(scope="module")
def lib():
    import bit_quantized_linear_vq_amd as vq
    return vq._lib


def norm(lib, **kw):
    a = dict(x=FAKE, res=FAKE, dt=BF16, m=4, k=128, ldx=128, ldr=128, w=FAKE, wdt=BF16, eps=1e-6, y=FAKE, ldy=128,
             h=FAKE, ldh=128)
    a.update(kw)
    return lib.vq_rmsnorm(a["x"], a["res"], a["dt"], a["m"], a["k"], a["ldx"], a["ldr"], a["w"], a["wdt"], a["eps"],
                          a["y"], a["ldy"], a["h"], a["ldh"], NULL)


@pytest.mark.parametrize("kw,want", [
    (dict(x=NULL), INVALID), (dict(y=NULL), INVALID), (dict(dt=F32), INVALID), (dict(dt=9), INVALID),
    (dict(m=-1), INVALID), (dict(k=0), INVALID), (dict(ldx=127), INVALID), (dict(ldr=100), INVALID),
    (dict(ldh=1), INVALID), (dict(ldy=5), INVALID), (dict(wdt=F16), INVALID), (dict(eps=-1e-9), INVALID),
    (dict(eps=NAN), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(k=32769, ldx=32769, ldr=32769, ldy=32769, ldh=32769), UNSUP),
    (dict(x=ctypes.c_void_p(0x10001)), SHAPE), (dict(y=ctypes.c_void_p(0x10001)), SHAPE),
    (dict(w=ctypes.c_void_p(0x10002), wdt=F32), SHAPE),
    (dict(m=0), OK), (dict(m=0, x=NULL, y=NULL, res=NULL, h=NULL), OK),
])
def test_rmsnorm_validation(lib, kw, want):
    assert norm(lib, **kw) == want


def normq(lib, **kw):
    a = dict(x=FAKE, res=FAKE, dt=BF16, m=4, k=128, ldx=128, ldr=128, w=FAKE, wdt=BF16, eps=1e-6, bits=8, bits_dev=NULL,
             gran=1, idx=NULL, n_out=0, st=NULL, codes=FAKE, scales=FAKE, h=FAKE, ldh=128)
    a.update(kw)
    return lib.vq_rmsnorm_quant(a["x"], a["res"], a["dt"], a["m"], a["k"], a["ldx"], a["ldr"], a["w"], a["wdt"],
                                a["eps"], a["bits"], a["bits_dev"], a["gran"], a["idx"], a["n_out"], a["st"],
                                a["codes"], a["scales"], a["h"], a["ldh"], NULL)


@pytest.mark.parametrize("kw,want", [
    (dict(codes=NULL), INVALID), (dict(scales=NULL), INVALID), (dict(n_out=-1), INVALID), (dict(n_out=2), INVALID),
    (dict(gran=5), INVALID), (dict(gran=2), INVALID), (dict(gran=0), UNSUP), (dict(bits=5), UNSUP),
    (dict(idx=FAKE, n_out=129, k=256, ldx=256, ldr=256, ldh=256), UNSUP), (dict(idx=FAKE, n_out=128), UNSUP),
    (dict(k=100), SHAPE), (dict(x=ODD), SHAPE), (dict(res=ODD), SHAPE), (dict(h=ODD), SHAPE), (dict(codes=ODD), SHAPE),
    (dict(ldx=130), SHAPE), (dict(ldr=132), SHAPE), (dict(ldh=129), SHAPE), (dict(m=0), OK),
])
def test_rmsnorm_quant_validation(lib, kw, want):
    assert normq(lib, **kw) == want


def packg(lib, **kw):
    a = dict(w=FAKE, dt=BF16, n=8, k=128, ldw=128, group=64, codes=FAKE, scales=FAKE)
    a.update(kw)
    return lib.vq_pack_weights_group(a["w"], a["dt"], a["n"], a["k"], a["ldw"], a["group"], a["codes"], a["scales"],
                                     NULL)


@pytest.mark.parametrize("kw,want", [
    (dict(w=NULL), INVALID), (dict(codes=NULL), INVALID), (dict(scales=NULL), INVALID), (dict(dt=F32), INVALID),
    (dict(n=0), INVALID), (dict(ldw=64), INVALID), (dict(group=48), UNSUP), (dict(group=0), UNSUP),
    (dict(k=96), SHAPE), (dict(w=ODD), SHAPE), (dict(codes=ODD), SHAPE), (dict(ldw=132), SHAPE),
    (dict(scales=ctypes.c_void_p(0x10001)), SHAPE),
])
def test_pack_group_validation(lib, kw, want):
    assert packg(lib, **kw) == want


def gemv(lib, **kw):
    a = dict(x=FAKE, dt=BF16, m=2, n=8, k=128, ldx=128, codes=FAKE, scales=FAKE, group=64, y=FAKE, out=BF16, ldy=8)
    a.update(kw)
    return lib.vq_w4_gemv(a["x"], a["dt"], a["m"], a["n"], a["k"], a["ldx"], a["codes"], a["scales"], a["group"],
                          a["y"], a["out"], a["ldy"], NULL)


@pytest.mark.parametrize("kw,want", [
    (dict(x=NULL), INVALID), (dict(codes=NULL), INVALID), (dict(scales=NULL), INVALID), (dict(y=NULL), INVALID),
    (dict(dt=F32), INVALID), (dict(out=7), INVALID), (dict(m=-1), INVALID), (dict(n=0), INVALID), (dict(k=0), INVALID),
    (dict(ldx=64), INVALID), (dict(ldy=7), INVALID), (dict(group=16), UNSUP), (dict(group=256, k=256, ldx=256), UNSUP),
    (dict(m=(1 << 20) + 1), UNSUP), (dict(n=(1 << 24) + 1, ldy=1 << 25), UNSUP),
    (dict(k=160, ldx=160), SHAPE), (dict(x=ODD), SHAPE), (dict(ldx=132), SHAPE), (dict(codes=ODD), SHAPE),
    (dict(y=ctypes.c_void_p(0x10002), out=F32), SHAPE), (dict(m=0, x=NULL, y=NULL), OK),
])
def test_gemv_validation(lib, kw, want):
    assert gemv(lib, **kw) == want


def experts(lib, **kw):
    a = dict(a=FAKE, sa=FAKE, b=FAKE, bits=8, sb=FAKE, off=FAKE, e=3, rows=NULL, m=10, t=10, n=32, k=128, y=FAKE,
             out=BF16, ldy=32)
    a.update(kw)
    return lib.vq_qgemm_experts(a["a"], a["sa"], a["b"], a["bits"], a["sb"], a["off"], a["e"], a["rows"], a["m"],
                                a["t"], a["n"], a["k"], a["y"], a["out"], a["ldy"], NULL)


@pytest.mark.parametrize("kw,want", [
    (dict(a=NULL), INVALID), (dict(sa=NULL), INVALID), (dict(b=NULL), INVALID), (dict(sb=NULL), INVALID),
    (dict(off=NULL), INVALID), (dict(y=NULL), INVALID), (dict(e=0), INVALID), (dict(t=-1), INVALID),
    (dict(t=11), INVALID), (dict(m=0, rows=FAKE), INVALID), (dict(n=0), INVALID), (dict(ldy=31), INVALID),
    (dict(out=3), INVALID), (dict(bits=6), UNSUP), (dict(bits=8 | 0x200), UNSUP), (dict(e=1025), UNSUP),
    (dict(t=(1 << 26) + 1, rows=FAKE), UNSUP), (dict(n=(1 << 20) + 1, ldy=1 << 21), UNSUP),
    (dict(k=1 << 25), UNSUP), (dict(k=100), SHAPE), (dict(k=133184), SHAPE), (dict(k=151040, bits=4), SHAPE),
    (dict(a=ODD), SHAPE), (dict(b=ODD), SHAPE), (dict(y=ctypes.c_void_p(0x10002), out=F32), SHAPE),
    (dict(t=0), OK), (dict(t=0, m=0, a=NULL, sa=NULL, y=NULL, rows=FAKE), OK),
])
def test_experts_validation(lib, kw, want):
    assert experts(lib, **kw) == want


def dense(lib, **kw):
    a = dict(x=FAKE, w=FAKE, dt=F16, off=FAKE, e=3, rows=NULL, m=10, t=10, n=32, k=128, ldx=128, ldw=128, es=4096,
             y=FAKE, out=F16, ldy=32)
    a.update(kw)
    return lib.vq_gemm_dense_experts(a["x"], a["w"], a["dt"], a["off"], a["e"], a["rows"], a["m"], a["t"], a["n"],
                                     a["k"], a["ldx"], a["ldw"], a["es"], a["y"], a["out"], a["ldy"], NULL)


@pytest.mark.parametrize("kw,want", [
    (dict(x=NULL), INVALID), (dict(w=NULL), INVALID), (dict(dt=F32), INVALID), (dict(ldx=64), INVALID),
    (dict(ldw=64), INVALID), (dict(es=-8), INVALID), (dict(k=96, ldx=96), SHAPE), (dict(ldx=132), SHAPE),
    (dict(ldw=130), SHAPE), (dict(es=4100), SHAPE), (dict(x=ODD), SHAPE), (dict(w=ODD), SHAPE), (dict(e=1025), UNSUP),
    (dict(t=0), OK),
])
def test_dense_experts_validation(lib, kw, want):
    assert dense(lib, **kw) == want
