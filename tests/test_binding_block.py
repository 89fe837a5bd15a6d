"""The binding's checks of the operators between the layers of a block, without a GPU: tensors that
have a device, a shape and no memory (torch's fake tensors) reach every check, and a call that
passes them all would reach the launch, which here only takes note."""
import os

import pytest
import torch
from torch._subclasses import FakeTensorMode

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "bit_quantized_linear_vq_amd", "libvq.so")

pytestmark = [pytest.mark.skipif(not os.path.exists(LIB), reason="libvq.so not built"),
              pytest.mark.filterwarnings("ignore")]

H, B, I8, I32 = torch.float16, torch.bfloat16, torch.int8, torch.int32


@pytest.fixture
def vq(monkeypatch):
    import bit_quantized_linear_vq_amd as m
    real = m._lib

    class Lib:
        launched = []

        def __getattr__(self, name):
            if name not in m._LAUNCHES:
                return getattr(real, name)
            return lambda *a: self.launched.append(name) or 0

    lib = Lib()
    lib.launched = []
    monkeypatch.setattr(m, "_lib", lib)
    monkeypatch.setattr(m, "_getdev", lambda: 0)
    monkeypatch.setattr(m, "_rawstream", lambda i: 0)
    with FakeTensorMode():
        yield m


def dev(*shape, dt=torch.float32):
    return torch.empty(shape, dtype=dt, device="cuda")


def refused(vq, error, f, *a, **kw):
    with pytest.raises(error):
        f(*a, **kw)
    assert vq._lib.launched == []


def gated(vq, quant=False, **kw):
    a = dict(branch=dev(6, 128, dt=B), residual=dev(6, 128, dt=B), sum_out=dev(6, 128, dt=B))
    a.update(dict(codes=dev(6, 128, dt=I8), scales=dev(6)) if quant else dict(y=dev(6, 128, dt=B)))
    a.update(kw)
    b, r = a.pop("branch"), a.pop("residual")
    return vq.vq_gated_norm_quant(b, r, a.pop("bits", 8), **a) if quant else vq.vq_gated_norm(b, r, **a)


def test_gated_calls_that_are_right_reach_the_launch(vq):
    wide = dev(3, 3 * 128)
    mods = dict(gate=wide[:, :128], mod_scale=wide[:, 128:256], mod_shift=wide[:, 256:])
    gated(vq)
    gated(vq, weight=dev(128), post="layer", post_weight=dev(128, dt=B), norm="layer", **mods)
    gated(vq, index=dev(6, dt=I32), gate=dev(4, 128, dt=B))
    gated(vq, branch=None, sum_out=None, mod_scale=dev(6, 128))
    gated(vq, True, **mods)
    gated(vq, True, gran="static", static_scale=dev(1), scales=dev(1))
    gated(vq, True, idx=dev(3, dt=I32), codes=dev(6, 192, dt=I8), scales=dev(6, 2))
    assert vq._lib.launched == ["vq_gated_norm"] * 4 + ["vq_gated_norm_quant"] * 3


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("error,kw", [
    (TypeError, lambda: dict(residual=torch.empty(6, 128, dtype=B))), (TypeError, lambda: dict(branch=dev(6, 128, dt=H))),
    (ValueError, lambda: dict(branch=dev(5, 128, dt=B))), (ValueError, lambda: dict(residual=dev(6 * 128, dt=B))),
    (ValueError, lambda: dict(residual=dev(128, 6, dt=B).t())), (ValueError, lambda: dict(sum_out=dev(6, 64, dt=B))),
    (TypeError, lambda: dict(sum_out=dev(6, 128))), (ValueError, lambda: dict(norm="none")), (ValueError, lambda: dict(norm=None)),
    (ValueError, lambda: dict(post="max")), (ValueError, lambda: dict(post_weight=dev(128))), (TypeError, lambda: dict(weight=dev(128, dt=H))),
    (ValueError, lambda: dict(weight=dev(129))), (ValueError, lambda: dict(weight=dev(64))), (TypeError, lambda: dict(gate=dev(2, 128, dt=H))),
    (ValueError, lambda: dict(gate=dev(128))), (ValueError, lambda: dict(gate=dev(2, 64))), (ValueError, lambda: dict(gate=dev(0, 128))),
    (ValueError, lambda: dict(gate=dev(4, 128))), (ValueError, lambda: dict(gate=dev(2, 128), mod_scale=dev(3, 128))),
    (ValueError, lambda: dict(gate=dev(2, 128), mod_shift=dev(2, 128, dt=B))), (TypeError, lambda: dict(mod_shift=torch.empty(2, 128))),
    (ValueError, lambda: dict(index=dev(6, dt=I32))), (TypeError, lambda: dict(gate=dev(2, 128), index=dev(6, dt=torch.int64))),
    (ValueError, lambda: dict(gate=dev(2, 128), index=dev(5, dt=I32))), (ValueError, lambda: dict(gate=dev(2, 128), index=dev(7, dt=I32))),
    (TypeError, lambda: dict(gate=dev(2, 128), index=torch.zeros(6, dtype=I32))),
    (ValueError, lambda: dict(gate=dev(1, 128).expand(2, 128))), (ValueError, lambda: dict(branch=None)),
    (ValueError, lambda: dict(branch=None, sum_out=None, gate=dev(2, 128))), (ValueError, lambda: dict(branch=None, sum_out=None, post="rms")),
])
def test_gated_refusals(vq, quant, error, kw):
    refused(vq, error, gated, vq, quant, **kw())


@pytest.mark.parametrize("error,kw", [
    (ValueError, lambda: dict(codes=dev(6, 64, dt=I8))), (TypeError, lambda: dict(codes=dev(6, 128, dt=torch.uint8))),
    (ValueError, lambda: dict(scales=dev(5))), (ValueError, lambda: dict(idx=dev(3, dt=I32), codes=dev(6, 192, dt=I8))),
    (TypeError, lambda: dict(idx=dev(3))), (TypeError, lambda: dict(bits_dev=dev(1))), (ValueError, lambda: dict(static_scale=dev(0))),
])
def test_gated_quant_refusals(vq, error, kw):
    refused(vq, error, gated, vq, True, **kw())


def test_gated_norm_refuses_another_output(vq):
    refused(vq, ValueError, gated, vq, y=dev(6, 127, dt=B))
    refused(vq, TypeError, gated, vq, y=dev(6, 128, dt=H))


def route(vq, **kw):
    a = dict(scores=dev(6, 16), top=2, offsets=dev(17, dt=I32), rows=dev(12, dt=I32), weights=dev(6, 2), experts=dev(6, 2, dt=I32),
             place=dev(6, 2, dt=I32), ws=dev(64, dt=I32))
    a.update(kw)
    return vq.vq_route_experts(**a)


def test_route_calls_that_are_right_reach_the_launch(vq):
    route(vq)
    route(vq, scores=dev(6, 16, dt=H), score="sigmoid", bias=dev(16), groups=4, top_groups=2, group_best=2)
    route(vq, scores=dev(6, 20)[:, :16])
    assert vq._lib.launched == ["vq_route_experts"] * 3


@pytest.mark.parametrize("error,kw", [
    (TypeError, lambda: dict(scores=torch.empty(6, 16))), (TypeError, lambda: dict(scores=dev(6, 16, dt=I32))),
    (ValueError, lambda: dict(scores=dev(96))), (ValueError, lambda: dict(scores=dev(16, 6).t())),
    (ValueError, lambda: dict(score="max")), (ValueError, lambda: dict(top=0)), (ValueError, lambda: dict(top=17)),
    (ValueError, lambda: dict(bias=dev(15))), (ValueError, lambda: dict(bias=dev(17))), (TypeError, lambda: dict(bias=dev(16, dt=H))),
    (ValueError, lambda: dict(offsets=dev(16, dt=I32))), (TypeError, lambda: dict(offsets=dev(17))),
    (ValueError, lambda: dict(rows=dev(6, 2, dt=I32))), (ValueError, lambda: dict(weights=dev(2, 6))),
    (ValueError, lambda: dict(weights=dev(2, 6).t())), (TypeError, lambda: dict(experts=dev(6, 2))), (TypeError, lambda: dict(ws=dev(64))),
    (TypeError, lambda: dict(place=torch.empty(6, 2, dtype=I32))), (ValueError, lambda: dict(scores=dev(65, 16), rows=None, weights=None, experts=None, place=None, ws=dev(15, dt=I32))),
])
def test_route_refusals(vq, error, kw):
    refused(vq, error, route, vq, **kw())


def combine(vq, **kw):
    a = dict(y=dev(12, 64, dt=B), place=dev(6, 2, dt=I32), weights=dev(6, 2), out=dev(6, 64, dt=B))
    a.update(kw)
    return vq.vq_combine_experts(**a)


def test_combine_calls_that_are_right_reach_the_launch(vq):
    combine(vq)
    combine(vq, residual=dev(6, 64, dt=B), gate=dev(3, 64))
    combine(vq, y=dev(12, 64), gate=dev(4, 64, dt=B), index=dev(6, dt=I32))
    combine(vq, y=dev(0, 64, dt=B))
    assert vq._lib.launched == ["vq_combine_experts"] * 4


@pytest.mark.parametrize("error,kw", [
    (TypeError, lambda: dict(y=dev(12, 64, dt=I32))), (ValueError, lambda: dict(y=dev(12 * 64, dt=B))),
    (TypeError, lambda: dict(place=dev(6, 2))), (ValueError, lambda: dict(place=dev(6, 3, dt=I32))),
    (ValueError, lambda: dict(place=dev(12, dt=I32), weights=dev(12))), (TypeError, lambda: dict(weights=dev(6, 2, dt=B))),
    (ValueError, lambda: dict(place=dev(6, 0, dt=I32), weights=dev(6, 0))),
    (ValueError, lambda: dict(residual=dev(6, 63, dt=B))), (TypeError, lambda: dict(residual=dev(6, 64))),
    (ValueError, lambda: dict(out=dev(5, 64, dt=B))), (TypeError, lambda: dict(out=dev(6, 64, dt=torch.int16))),
    (ValueError, lambda: dict(gate=dev(4, 64))), (ValueError, lambda: dict(index=dev(6, dt=I32))),
    (TypeError, lambda: dict(gate=dev(2, 64, dt=H))), (TypeError, lambda: dict(out=torch.empty(6, 64, dtype=B))),
])
def test_combine_refusals(vq, error, kw):
    refused(vq, error, combine, vq, **kw())


def lowrank(vq, **kw):
    a = dict(base=dev(6, 48, dt=B), x=dev(6, 128, dt=B), down=dev(3, 16, 128, dt=B), up=dev(3, 48, 16, dt=B), index=dev(6, dt=I32),
             scales=dev(3), out=dev(6, 48, dt=B), ws=dev(4096))
    a.update(kw)
    return vq.vq_lowrank_add(**a)


def test_lowrank_calls_that_are_right_reach_the_launch(vq):
    lowrank(vq)
    lowrank(vq, base=dev(6, 48), out=dev(6, 50)[:, :48], scales=None)
    lowrank(vq, x=dev(0, 128, dt=B), base=dev(0, 48, dt=B), out=dev(0, 48, dt=B), index=dev(0, dt=I32))
    assert vq._lib.launched == ["vq_lowrank_add"] * 3


@pytest.mark.parametrize("error,kw", [
    (TypeError, lambda: dict(x=dev(6, 128))), (ValueError, lambda: dict(x=dev(128, 6, dt=B).t())),
    (TypeError, lambda: dict(base=dev(6, 48, dt=H))), (ValueError, lambda: dict(base=dev(5, 48, dt=B))),
    (TypeError, lambda: dict(down=dev(3, 16, 128, dt=H))), (ValueError, lambda: dict(down=dev(3, 16, 64, dt=B))),
    (ValueError, lambda: dict(down=dev(48, 128, dt=B))), (ValueError, lambda: dict(up=dev(3, 16, 48, dt=B))),
    (ValueError, lambda: dict(up=dev(2, 48, 16, dt=B))), (ValueError, lambda: dict(up=dev(3, 16, 48, dt=B).transpose(1, 2))),
    (TypeError, lambda: dict(index=dev(6, dt=torch.int64))), (ValueError, lambda: dict(index=dev(5, dt=I32))),
    (ValueError, lambda: dict(index=dev(7, dt=I32))), (TypeError, lambda: dict(index=torch.zeros(6, dtype=I32))),
    (ValueError, lambda: dict(scales=dev(2))), (ValueError, lambda: dict(scales=dev(4))), (TypeError, lambda: dict(scales=dev(3, dt=B))),
    (TypeError, lambda: dict(out=dev(6, 48))), (ValueError, lambda: dict(out=dev(6, 47, dt=B))),
    (ValueError, lambda: dict(ws=dev(8))), (TypeError, lambda: dict(ws=dev(4096, dt=B))),
])
def test_lowrank_refusals(vq, error, kw):
    refused(vq, error, lowrank, vq, **kw())


def test_operands_without_rows_may_have_any_strides(vq):
    """torch gives a tensor without elements strides that say nothing."""
    x = torch.empty_strided((0, 128), (1, 7), dtype=B, device="cuda")
    lowrank(vq, x=x, base=dev(0, 48, dt=B), out=dev(0, 48, dt=B), index=dev(0, dt=I32))
    gated(vq, branch=x, residual=x, y=x, sum_out=x)
    route(vq, scores=torch.empty_strided((0, 16), (1, 3), device="cuda"), rows=None, weights=None, experts=None, place=None)
    assert len(vq._lib.launched) == 3
