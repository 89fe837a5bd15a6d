"""The binding's checks of device tensors, without a GPU: tensors that have a device, a shape and
no memory (torch's fake tensors) reach every check, and a call that passes them all would
reach the launch, which here only takes note."""
import gc
import os
import weakref

import pytest
import torch
from torch._subclasses import FakeTensorMode

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "bit_quantized_linear_vq_amd", "libvq.so")

pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libvq.so not built")


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
    monkeypatch.setattr(m, "_stream", lambda t: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 0)
    with FakeTensorMode():
        yield m


def launched(vq):
    return list(vq._lib.launched)


def dev(*shape, dt=torch.float32):
    return torch.empty(shape, dtype=dt, device="cuda")


def experts(vq, bits=8, m=6, e=2, n=32, k=128, **kw):
    rb = k if bits & 15 == 8 else k // 2
    wt = torch.int8 if bits & 15 == 8 else torch.uint8
    a = dict(a=dev(m, k, dt=torch.int8), sa=dev(m), b=dev(e * n, rb, dt=wt), sb=dev(e * n), b_bits=bits,
             offsets=dev(e + 1, dt=torch.int32), y=dev(m, n, dt=torch.bfloat16))
    a.update(kw)
    return vq.vq_qgemm_experts(**a)


@pytest.mark.filterwarnings("ignore")
def test_a_call_that_is_right_reaches_the_launch(vq):
    experts(vq)
    experts(vq, 4)
    experts(vq, b=dev(2, 64, 64, dt=torch.int8))
    experts(vq, 8 | vq.VQ_W_KBLOCK, b=dev(2, 64, 64, dt=torch.int8))
    assert launched(vq) == ["vq_qgemm_experts"] * 4


@pytest.mark.parametrize("bits", [8, 4])
def test_the_piece_flag_in_the_width_passes_no_check_by(vq, bits):
    """With it the library would read row-major codes, or codes of another shape, as pieces."""
    flag, wt = bits | vq.VQ_W_KBLOCK, torch.int8 if bits == 8 else torch.uint8
    with pytest.raises(ValueError):
        experts(vq, flag)
    with pytest.raises(ValueError):
        experts(vq, flag, b=dev(1, 64, 64 if bits == 8 else 32, dt=wt))
    with pytest.raises(TypeError):
        experts(vq, flag, b=torch.empty(2, 64, 64, dtype=wt))
    a, sa, sb = dev(6, 128, dt=torch.int8), dev(6), dev(32)
    with pytest.raises(ValueError):
        vq.vq_qgemm_dequant(a, sa, dev(32, 16, dt=wt), sb, flag, y=dev(6, 32, dt=torch.bfloat16), ws=False)
    with pytest.raises(ValueError):
        vq.vq_qgemm_dequant(a, sa, dev(5, 32, 64, dt=wt), sb, flag, y=dev(6, 32, dt=torch.bfloat16), ws=False)
    with pytest.raises(TypeError):
        vq.vq_qgemm_dequant(a, sa, torch.empty(2, 32, 64, dtype=wt), sb, flag, y=dev(6, 32, dt=torch.bfloat16), ws=False)
    assert not launched(vq)


@pytest.mark.parametrize("kw", [
    dict(sa=(6, 2)), dict(sa=(12,)), dict(sb=(64, 2)), dict(sb=(128,)), dict(sa=(6, 2), sb=(64, 2)), dict(sa=(5,)), dict(sb=(63,)),
])
def test_scales_of_two_partitions_are_refused(vq, kw):
    """The codes of an outlier partition have two scales a row: the experts take one."""
    with pytest.raises(ValueError):
        experts(vq, **{n: dev(*shape) for n, shape in kw.items()})
    assert not launched(vq)


def test_operands_with_an_outlier_partition_do_not_fit_the_experts(vq):
    """As the quantizers return them: codes [M x kp], scales [M x 2]."""
    idx, x, w = dev(3, dt=torch.int32), dev(6, 128, dt=torch.bfloat16), dev(64, 128, dt=torch.bfloat16)
    a, sa = vq.vq_rmsnorm_quant(x, None, 8, idx=idx)
    b, sb = vq.vq_pack_weights(w, 8, idx=idx)
    off = dev(3, dt=torch.int32)
    vq._lib.launched.clear()
    with pytest.raises(ValueError, match="one partition"):
        vq.vq_qgemm_experts(a, sa, b, sb, 8, off)
    with pytest.raises(ValueError, match="one partition"):
        vq.vq_qgemm_experts(a, dev(6), b, sb, 8, off)
    assert not launched(vq)


@pytest.mark.filterwarnings("ignore")
def test_prepared_calls_hold_every_tensor_that_they_address(vq):
    """A function's own tensors too: what it drops when it returns is still written to by the
    recorded launches."""
    w = dev(64, 128, dt=torch.bfloat16)
    gone = []

    def f(x):
        c, s, h = vq.vq_rmsnorm_quant(x, None, 8, residual=x[:, :128])
        n = vq.vq_rmsnorm(x, dev(128).to(torch.bfloat16))
        b, sb = vq.vq_pack_weights(w, 8)
        gone.extend(weakref.ref(t) for t in (c, s, h, n, b, sb))
        return vq.vq_qgemm_experts(c, s, b, sb, 8, dev(3, dt=torch.int32)), vq.vq_gemm_dense_experts(
            n, w.view(2, 32, 128), dev(3, dt=torch.int32))

    launch, out = vq.prepare(f, dev(6, 128, dt=torch.bfloat16))
    gc.collect()
    assert [r() is None for r in gone] == [False] * len(gone)
    assert not launched(vq) and len(out) == 2
    launch()
    assert launched(vq) == ["vq_rmsnorm_quant", "vq_rmsnorm", "vq_pack_weights", "vq_qgemm_experts", "vq_gemm_dense_experts"]
    del launch, out
    gc.collect()
    assert all(r() is None for r in gone)


@pytest.mark.filterwarnings("ignore")
def test_prepared_calls_run_on_the_device_of_their_tensors(vq, monkeypatch):
    """As the calls themselves do: with that device current, on its current stream."""
    current, streams = [0], []

    def exchange(i):
        prev, current[0] = current[0], i
        return prev
    monkeypatch.setattr(vq, "_getdev", lambda: current[0])
    monkeypatch.setattr(torch._C, "_cuda_exchangeDevice", exchange)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: streams.append((i, current[0])) or 70 + i)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    x = torch.empty(6, 128, dtype=torch.bfloat16, device="cuda:1")
    launch, y = vq.prepare(lambda: vq.vq_rmsnorm(x, None))  # no tensor among the arguments
    streams.clear()
    launch()
    assert streams == [(1, 1)] and current == [0] and y.get_device() == 1
    x0 = dev(6, 128, dt=torch.bfloat16)
    with pytest.raises(ValueError, match="device"):
        vq.prepare(lambda: (vq.vq_rmsnorm(x, None), vq.vq_rmsnorm(x0, None)))
