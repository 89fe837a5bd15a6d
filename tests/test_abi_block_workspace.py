"""Scratch sizes of the routing and of the low-rank adapters, without a GPU: a buffer sized for the largest
call that a program makes serves every smaller one, since the calls take no size to check."""
import os
import random

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "bit_quantized_linear_vq_amd", "libvq.so")

pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libvq.so not built")


@pytest.fixture(scope="module")
def lib():
    import bit_quantized_linear_vq_amd as m
    return m._lib


ROWS = sorted({1, 2, 3, 4, 5, 15, 16, 17, 63, 64, 65, 255, 256, 257, 512, 513, 1000, 1023, 1024, 4000, 4096, 4097, 5159, 8191, 8192,
               8193, 12000, 13439, 15999, 16000, 16384, 16385, 17776, 32768, 100000, 1 << 20, 1 << 26})
ADAPTERS, RANKS, KS = [1, 2, 3, 4, 5, 8, 16, 31, 32, 33, 1000, 1 << 20], list(range(8, 129, 8)), [64, 512, 1024, 1920, 2048, 4096, 8192, 9088, 1 << 24]


def test_adapters_scratch_never_shrinks(lib):
    n = lib.vq_lowrank_workspace_elems
    for r in RANKS:
        for k in KS:
            for a in ADAPTERS:
                sizes = [n(m, a, r, k) for m in ROWS]
                assert sizes == sorted(sizes), (a, r, k)
    for m in ROWS:
        for k in KS:
            for r in RANKS:
                sizes = [n(m, a, r, k) for a in ADAPTERS]
                assert sizes == sorted(sizes), (m, r, k)
            for a in ADAPTERS:
                sizes = [n(m, a, r, k) for r in RANKS]
                assert sizes == sorted(sizes), (m, a, k)
        for a in ADAPTERS:
            for r in RANKS:
                sizes = [n(m, a, r, k) for k in KS]
                assert sizes == sorted(sizes), (m, a, r)


def test_adapters_scratch_of_a_largest_call_is_enough(lib):
    n = lib.vq_lowrank_workspace_elems
    rng = random.Random(1)
    for _ in range(5000):
        most = (rng.randint(1, 40000), rng.randint(1, 40), 8 * rng.randint(1, 16), 64 * rng.randint(1, 200))
        less = (rng.randint(1, most[0]), rng.randint(1, most[1]), 8 * rng.randint(1, most[2] // 8), 64 * rng.randint(1, most[3] // 64))
        assert n(*less) <= n(*most), (less, most)


def test_routing_scratch_never_shrinks(lib):
    n = lib.vq_route_experts_workspace_elems
    experts = [1, 2, 8, 16, 63, 64, 65, 96, 128, 160, 161, 255, 256, 257, 360, 512, 513, 1023, 1024]
    for e in experts:
        sizes = [n(m, e) for m in range(3000)] + [n(m, e) for m in ROWS if m >= 3000]
        assert sizes == sorted(sizes), e
    for m in ROWS:
        sizes = [n(m, e) for e in experts]
        assert sizes == sorted(sizes), m


def test_scratch_stays_small(lib):
    """A few rows need a few rows' worth, and many no more than their own t."""
    n = lib.vq_lowrank_workspace_elems
    assert n(1, 4, 64, 1920) <= 8 * 64 and n(48, 12, 16, 4096) <= 48 * 16 * 8
    for m in (32768, 100000, 1 << 20):
        assert n(m, 5, 32, 8192) == m * 32
    r = lib.vq_route_experts_workspace_elems
    assert r(1 << 26, 1024) * 4 <= 4 << 20
