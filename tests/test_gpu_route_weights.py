"""Weights of the routing against the definition in 64 bits (oracle/router.py): float64 values rounded once, so
within half a step of float32, 2^-24, and what E float64 operations may add, E 2^-50."""
import numpy as np
import pytest
import torch

from oracle import router

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def vq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_quantized_linear_vq_amd as m
    return m


def scores(m, e, seed=0, masked=0.0):
    rng = np.random.default_rng([m, e, seed])
    x = (1.5 * rng.standard_normal((m, e))).astype(np.float32)
    x[rng.random((m, e)) < masked] = -np.inf
    return torch.from_numpy(x)


def check(got, x, top, scale=1.0, bias=None, top_groups=None, group_best=1, **how):
    torch.cuda.synchronize()
    off, rows, w, ch, place = (t.cpu().numpy() for t in got)
    want = router.route(x.double().numpy(), top, bias=None if bias is None else bias.double().numpy(), keep=top_groups, best=group_best, **how)
    assert np.array_equal(ch, want[3]) and np.array_equal(off, want[0]) and np.array_equal(rows, want[1]) and np.array_equal(place, want[4])
    exact = want[2] * scale
    assert np.all(np.abs(w.astype(np.float64) - exact) <= (2.0 ** -24 + x.shape[1] * 2.0 ** -50) * np.abs(exact) + 2.0 ** -150)
    return w


@pytest.mark.parametrize("m,e,top,how", [
    (3, 7, 2, {}), (300, 16, 3, {}), (500, 160, 6, {}), (200, 256, 8, dict(groups=8, top_groups=3)), (150, 300, 5, {}), (100, 1024, 9, {}),
    (40, 64, 4, {}), (400, 96, 4, dict(groups=4, top_groups=2)),
])
def test_a_softmax_that_is_not_renormalised(vq, m, e, top, how):
    for masked in (0.0, 0.1):
        x = scores(m, e, masked=masked)
        check(vq.vq_route_experts(x.to(DEV), top, renorm=False, **how), x, top, renorm=False, **how)


@pytest.mark.parametrize("scale", [0.1, 2.446, 1.0 / 3.0, -0.7])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_a_scale_that_float32_does_not_hold(vq, renorm, score, scale):
    for m in (20, 400):
        x = scores(m, 48)
        check(vq.vq_route_experts(x.to(DEV), 5, score=score, renorm=renorm, scale=scale), x, 5, scale, score=score, renorm=renorm)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("how", [{}, dict(groups=4, top_groups=2, group_best=2)])
def test_an_expert_closed_by_its_bias_is_never_chosen_and_keeps_its_share(vq, how, renorm, score):
    """A bias moves the choice alone: the others' p are what they are without it."""
    m, e = 200, 40
    x = scores(m, e)
    bias = torch.linspace(-0.1, 0.1, e)
    bias[::7] = -float("inf")
    got = vq.vq_route_experts(x.to(DEV), 4, score=score, renorm=renorm, bias=bias.to(DEV), **how)
    w = check(got, x, 4, score=score, renorm=renorm, bias=bias, **how)
    ch = got[3].cpu().long()
    assert not torch.isin(ch, torch.arange(0, e, 7)).any()
    if not renorm:
        p = torch.softmax(x.double(), 1) if score == "softmax" else torch.sigmoid(x.double())
        assert np.allclose(w, torch.gather(p, 1, ch).numpy(), rtol=2.0 ** -23, atol=0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("m", [3, 20, 150])
@pytest.mark.parametrize("e,top,how", [
    (161, 6, {}), (192, 8, dict(groups=8, top_groups=4, group_best=2)), (200, 8, {}), (224, 8, dict(groups=7, top_groups=3)),
    (256, 8, {}), (256, 8, dict(groups=8, top_groups=4, group_best=2)), (256, 32, dict(groups=64, top_groups=20)),
    (513, 5, {}), (600, 8, dict(groups=6, top_groups=2, group_best=2)), (1024, 32, {}), (1024, 9, dict(groups=64, top_groups=9, group_best=2)),
])
def test_many_experts_chosen_by_p(vq, e, top, how, m, score):
    x = scores(m, e, masked=0.1)
    bias = 0.05 * torch.randn(e, generator=torch.Generator().manual_seed(e))
    for renorm in (True, False):
        check(vq.vq_route_experts(x.to(DEV), top, score=score, bias=bias.to(DEV), renorm=renorm, **how), x, top, score=score, bias=bias,
              renorm=renorm, **how)
    if how.get("group_best") == 2:
        check(vq.vq_route_experts(x.to(DEV), top, score=score, **how), x, top, score=score, **how)
