"""C-ABI checks, without a GPU, of the operators between the layers of a block: invalid arguments
get the documented status before any HIP call, and calls with no rows return without one."""
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
FAKE, ODD, BYTE = 0x10000, 0x10008, 0x10001
NULL = None
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def vq():
    import bit_quantized_linear_vq_amd as m
    return m


GATED = dict(y=FAKE, h=FAKE, dt=BF16, m=4, k=128, ldy=128, ldh=128, post=1, pw=FAKE, pwdt=F32, alpha=1.0, gate=FAKE,
             scale=FAKE, shift=FAKE, ldg=128, ldsc=128, ldsh=128, index=NULL, sets=2, mdt=F32, norm=2, w=FAKE, wdt=BF16,
             eps=1e-6, n=FAKE, ldn=128, s=FAKE, lds=128, mod=True)


def head(vq, a):
    mod = vq.Modulation(a["gate"], a["scale"], a["shift"], a["ldg"], a["ldsc"], a["ldsh"], a["index"], a["sets"], a["mdt"], 0)
    return (a["y"], a["h"], a["dt"], a["m"], a["k"], a["ldy"], a["ldh"], a["post"], a["pw"], a["pwdt"], a["alpha"],
            ctypes.byref(mod) if a["mod"] else None, a["norm"], a["w"], a["wdt"], a["eps"])


def gated(vq, **kw):
    a = {**GATED, **kw}
    return vq._lib.vq_gated_norm(*head(vq, a), a["n"], a["ldn"], a["s"], a["lds"], NULL)


NO_BRANCH = dict(y=NULL, s=NULL, post=0, pw=NULL, gate=NULL)
BAD_GATED = [
    (dict(h=NULL), INVALID), (dict(s=NULL), INVALID), (dict(dt=F32), INVALID), (dict(m=-1), INVALID), (dict(k=0), INVALID),
    (dict(ldy=127), INVALID), (dict(ldh=64), INVALID), (dict(lds=127), INVALID), (dict(pwdt=F16), INVALID),
    (dict(wdt=F16), INVALID), (dict(norm=0), INVALID), (dict(norm=3), INVALID), (dict(post=5), INVALID),
    (dict(post=0), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=NAN), INVALID), (dict(alpha=INF), INVALID),
    (dict(alpha=NAN), INVALID), (dict(alpha=1e300), INVALID), (dict(mdt=F16), INVALID), (dict(sets=0), INVALID),
    (dict(sets=-2), INVALID), (dict(ldg=127), INVALID), (dict(ldsc=127), INVALID), (dict(ldsh=0), INVALID),
    ({**NO_BRANCH, "s": FAKE}, INVALID), ({**NO_BRANCH, "post": 1}, INVALID), ({**NO_BRANCH, "gate": FAKE}, INVALID),
    ({**NO_BRANCH, "pw": FAKE}, INVALID),
    (dict(sets=3), SHAPE), (dict(gate=0x10002), SHAPE), (dict(scale=BYTE, mdt=BF16), SHAPE), (dict(shift=0x10003), SHAPE),
    (dict(index=0x10002), SHAPE), (dict(h=BYTE), SHAPE), (dict(y=BYTE), SHAPE), (dict(s=BYTE), SHAPE),
    (dict(w=BYTE), SHAPE), (dict(pw=0x10002), SHAPE),
]


@pytest.mark.parametrize("kw,want", BAD_GATED + [
    (dict(n=NULL), INVALID), (dict(ldn=100), INVALID), (dict(n=BYTE), SHAPE),
    (dict(k=32769, ldy=32769, ldh=32769, ldn=32769, lds=32769), UNSUP),
    (dict(m=0), OK), (dict(m=0, y=NULL, h=NULL, n=NULL, s=NULL, mod=False, post=0, pw=NULL), OK),
])
def test_gated_norm_validation(vq, kw, want):
    assert gated(vq, **kw) == want


def gatedq(vq, **kw):
    a = {**GATED, **dict(bits=8, bits_dev=NULL, gran=1, idx=NULL, n_out=0, st=NULL, codes=FAKE, scales=FAKE), **kw}
    return vq._lib.vq_gated_norm_quant(*head(vq, a), a["bits"], a["bits_dev"], a["gran"], a["idx"], a["n_out"], a["st"],
                                       a["codes"], a["scales"], a["s"], a["lds"], NULL)


@pytest.mark.parametrize("kw,want", BAD_GATED + [
    (dict(codes=NULL), INVALID), (dict(scales=NULL), INVALID), (dict(n_out=-1), INVALID), (dict(n_out=2), INVALID),
    (dict(gran=5), INVALID), (dict(gran=2), INVALID), (dict(gran=0), UNSUP), (dict(bits=5), UNSUP),
    (dict(idx=FAKE, n_out=128), UNSUP), (dict(k=100), SHAPE), (dict(h=ODD), SHAPE), (dict(y=ODD), SHAPE), (dict(s=ODD), SHAPE),
    (dict(codes=ODD), SHAPE), (dict(ldy=130), SHAPE), (dict(ldh=132), SHAPE), (dict(lds=129), SHAPE), (dict(m=0), OK),
])
def test_gated_norm_quant_validation(vq, kw, want):
    assert gatedq(vq, **kw) == want


def route(vq, **kw):
    a = {**dict(x=FAKE, dt=F32, m=4, e=16, ldx=16, score=0, bias=FAKE, groups=4, keep=2, best=2, top=3, renorm=1, scale=1.0,
                off=FAKE, rows=FAKE, w=FAKE, ch=FAKE, place=FAKE, ws=FAKE), **kw}
    return vq._lib.vq_route_experts(a["x"], a["dt"], a["m"], a["e"], a["ldx"], a["score"], a["bias"], a["groups"], a["keep"],
                                    a["best"], a["top"], a["renorm"], a["scale"], a["off"], a["rows"], a["w"], a["ch"],
                                    a["place"], a["ws"], NULL)


@pytest.mark.parametrize("kw,want", [
    (dict(x=NULL), INVALID), (dict(dt=7), INVALID), (dict(m=-1), INVALID), (dict(e=0), INVALID), (dict(ldx=15), INVALID),
    (dict(score=2), INVALID), (dict(score=-1), INVALID), (dict(off=NULL), INVALID), (dict(rows=NULL), INVALID),
    (dict(w=NULL), INVALID), (dict(ch=NULL), INVALID), (dict(place=NULL), INVALID), (dict(m=65, ws=NULL), INVALID),
    (dict(groups=0), INVALID), (dict(groups=3), INVALID), (dict(keep=0), INVALID), (dict(keep=5), INVALID),
    (dict(best=0), INVALID), (dict(best=3), INVALID), (dict(groups=16, keep=8), INVALID), (dict(top=0), INVALID),
    (dict(top=9), INVALID), (dict(scale=INF), INVALID), (dict(scale=NAN), INVALID),
    (dict(e=1028, ldx=1028), UNSUP), (dict(e=256, ldx=256, top=33), UNSUP), (dict(e=512, ldx=512, groups=128), UNSUP),
    (dict(m=1 << 25), UNSUP), (dict(m=1 << 62), UNSUP),
    (dict(x=0x10002), SHAPE), (dict(bias=0x10002), SHAPE), (dict(off=0x10002), SHAPE), (dict(rows=BYTE), SHAPE),
    (dict(w=0x10002), SHAPE), (dict(ch=0x10002), SHAPE), (dict(place=0x10003), SHAPE), (dict(ws=0x10002), SHAPE),
])
def test_route_validation(vq, kw, want):
    assert route(vq, **kw) == want


def test_route_workspace(vq):
    n = vq._lib.vq_route_experts_workspace_elems
    assert n(-1, 8) == n(8, 0) == n(8, 1025) == n((1 << 26) + 1, 8) == 0
    assert n(0, 8) == n(64, 64) == n(16, 256) == n(4, 1024) == 0 and n(17, 256) > 0 and n(5, 1024) > 0 and n(65, 1) > 0 and n(1 << 26, 1024) >= 1024


def combine(vq, **kw):
    a = {**dict(y=FAKE, ydt=BF16, rows=8, ldy=64, place=FAKE, w=FAKE, m=4, n=64, top=2, res=FAKE, ldr=64, out=FAKE, odt=BF16,
                ldo=64, mod=True, gate=FAKE, scale=NULL, shift=NULL, ldg=64, ldsc=64, ldsh=64, index=NULL, sets=2, mdt=F32), **kw}
    mod = vq.Modulation(a["gate"], a["scale"], a["shift"], a["ldg"], a["ldsc"], a["ldsh"], a["index"], a["sets"], a["mdt"], 0)
    return vq._lib.vq_combine_experts(a["y"], a["ydt"], a["rows"], a["ldy"], a["place"], a["w"], a["m"], a["n"], a["top"],
                                      a["res"], a["ldr"], ctypes.byref(mod) if a["mod"] else None, a["out"], a["odt"],
                                      a["ldo"], NULL)


@pytest.mark.parametrize("kw,want", [
    (dict(y=NULL), INVALID), (dict(ydt=3), INVALID), (dict(odt=5), INVALID), (dict(rows=-1), INVALID), (dict(ldy=63), INVALID),
    (dict(place=NULL), INVALID), (dict(w=NULL), INVALID), (dict(m=-1), INVALID), (dict(n=0), INVALID), (dict(top=0), INVALID),
    (dict(ldr=63), INVALID), (dict(out=NULL), INVALID), (dict(ldo=10), INVALID), (dict(scale=FAKE), INVALID),
    (dict(shift=FAKE), INVALID), (dict(mdt=F16), INVALID), (dict(sets=0), INVALID), (dict(ldg=63), INVALID),
    (dict(odt=F16), UNSUP), (dict(top=33), UNSUP), (dict(m=(1 << 26) + 1), UNSUP), (dict(rows=(1 << 26) + 1), UNSUP),
    (dict(n=(1 << 20) + 1, ldy=1 << 21, ldr=1 << 21, ldo=1 << 21), UNSUP),
    (dict(sets=3), SHAPE), (dict(y=BYTE), SHAPE), (dict(res=BYTE), SHAPE), (dict(out=0x10002, odt=F32), SHAPE),
    (dict(place=0x10002), SHAPE), (dict(w=0x10002), SHAPE), (dict(gate=0x10002), SHAPE),
    (dict(m=0), OK), (dict(m=0, y=NULL, place=NULL, w=NULL, out=NULL, res=NULL, mod=False), OK),
])
def test_combine_validation(vq, kw, want):
    assert combine(vq, **kw) == want


def lowrank(vq, **kw):
    a = {**dict(x=FAKE, dt=BF16, m=4, n=32, k=128, ldx=128, down=FAKE, up=FAKE, ad=3, r=16, index=FAKE, scale=FAKE, base=FAKE,
                ldb=32, out=FAKE, odt=BF16, ldo=32, ws=FAKE), **kw}
    return vq._lib.vq_lowrank_add(a["x"], a["dt"], a["m"], a["n"], a["k"], a["ldx"], a["down"], a["up"], a["ad"], a["r"],
                                  a["index"], a["scale"], a["base"], a["ldb"], a["out"], a["odt"], a["ldo"], a["ws"], NULL)


@pytest.mark.parametrize("kw,want", [
    (dict(x=NULL), INVALID), (dict(dt=F32), INVALID), (dict(odt=F16), INVALID), (dict(odt=9), INVALID), (dict(m=-1), INVALID),
    (dict(n=0), INVALID), (dict(k=0), INVALID), (dict(ldx=64), INVALID), (dict(ldb=31), INVALID), (dict(ldo=0), INVALID),
    (dict(down=NULL), INVALID), (dict(up=NULL), INVALID), (dict(ad=0), INVALID), (dict(r=0), INVALID), (dict(index=NULL), INVALID),
    (dict(base=NULL), INVALID), (dict(out=NULL), INVALID), (dict(ws=NULL), INVALID),
    (dict(r=136), UNSUP), (dict(ad=(1 << 20) + 1), UNSUP), (dict(n=(1 << 24) + 1, ldb=1 << 25, ldo=1 << 25), UNSUP),
    (dict(k=(1 << 24) + 64, ldx=1 << 25), UNSUP), (dict(m=(1 << 31) - 1, n=1 << 20, ldb=1 << 20, ldo=1 << 20), UNSUP),
    (dict(m=1 << 29), UNSUP), (dict(m=1 << 20, n=1 << 17, ldb=1 << 17, ldo=1 << 17), UNSUP),
    (dict(r=12), SHAPE), (dict(k=96, ldx=96), SHAPE), (dict(ldx=132), SHAPE), (dict(x=ODD), SHAPE), (dict(down=ODD), SHAPE),
    (dict(up=ODD), SHAPE), (dict(ws=ODD), SHAPE), (dict(index=0x10002), SHAPE), (dict(scale=0x10002), SHAPE),
    (dict(base=BYTE), SHAPE), (dict(out=0x10002, odt=F32), SHAPE),
    (dict(m=0), OK), (dict(m=0, x=NULL, index=NULL, base=NULL, out=NULL), OK),
])
def test_lowrank_validation(vq, kw, want):
    assert lowrank(vq, **kw) == want


def test_lowrank_workspace(vq):
    n = vq._lib.vq_lowrank_workspace_elems
    assert n(-1, 1, 8, 64) == n(1, 0, 8, 64) == n(1, 1, 12, 64) == n(1, 1, 136, 64) == n(1, 1, 8, 0) == 0
    for m in (0, 1, 17, 5000, 1 << 20):
        for r in (8, 128):
            assert n(m, 4, r, 4096) >= max(m, 1) * r
