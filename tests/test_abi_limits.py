"""C-ABI limits of the norm, the group-scaled product and the experts that come from the kernels'
32-bit arithmetic, without a GPU: sizes above them get a status before any HIP call."""
import ctypes
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "bit_quantized_linear_vq_amd", "libvq.so")

# Fake device addresses: only where no GPU could be reached by a call that does not reject them.
pytestmark = [
    pytest.mark.skipif(not os.path.exists(LIB), reason="libvq.so not built"),
    pytest.mark.skipif(os.path.exists("/dev/kfd"), reason="a GPU is present: fake device addresses must not reach it"),
]

OK, INVALID, SHAPE, UNSUP, HIP = range(5)
BF16 = 1
FAKE = ctypes.c_void_p(0x10000)


@pytest.fixture(scope="module")
def lib():
    import bit_quantized_linear_vq_amd as vq
    return vq._lib


@pytest.mark.parametrize("k,m,want", [
    (2 ** 30, 0, OK), (2 ** 30 + 128, 0, UNSUP), (2 ** 30 + 128, 1, UNSUP), (2 ** 31 - 128, 1, UNSUP), (2 ** 31 - 32, 1, UNSUP),
])
def test_group_product_channels(lib, k, m, want):
    """A piece of 128 channels past the end of the last ones would not be counted in 32 bits."""
    assert lib.vq_w4_gemv(FAKE, BF16, m, 8, k, k, FAKE, FAKE, 32, FAKE, BF16, 8, None) == want
