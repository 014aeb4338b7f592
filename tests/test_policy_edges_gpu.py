"""policy_loss where a ratio is undefined or beyond float32, on every kernel:
a row to a warp, to a CTA, to a cluster, and the ring."""

import pytest
import torch

from tests.test_policy_loss_gpu import check, reference

pytestmark = pytest.mark.gpu

dev = torch.device("cuda")
BF, F32 = torch.bfloat16, torch.float32

SHAPES = [(300, 64, F32), (300, 2000, BF), (6, 5000, BF), (700, 12296, BF), (700, 16392, F32)]


def batch(T, V, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    z = torch.randn(T, V, device=dev, generator=g).to(dtype)
    a = torch.randint(V, (T,), device=dev, generator=g)
    lp = torch.log_softmax(z.double(), 1)[torch.arange(T, device=dev), a].float()
    return z, a, lp - 0.05, 0.5 + torch.rand(T, device=dev, generator=g), torch.full((T,), 1.0 / T, device=dev), lp


@pytest.mark.parametrize("T,V,dtype", SHAPES)
@pytest.mark.parametrize("which", ["old_logp", "advantage"])
@pytest.mark.parametrize("beta", [0.0, 0.1])
def test_undefined_ratio_shows_in_the_gradient(lib, T, V, dtype, which, beta):
    """A NaN old log-probability or advantage of a live token makes its loss
    NaN, and so its gradient: a step on a gradient of zeros would hide it."""
    z, a, old, adv, w, ref = batch(T, V, dtype, T + V)
    clean = lib.policy_loss(z, a, old, adv, w, ref_logp=ref, beta=beta)
    bad = [0, T // 2, T - 1]
    (old if which == "old_logp" else adv)[bad] = float("nan")
    loss, lp, dz = lib.policy_loss(z, a, old, adv, w, ref_logp=ref, beta=beta)
    assert loss.isnan().all() and torch.equal(lp, clean[1])
    assert dz[bad].isnan().all()
    rest = torch.ones(T, dtype=torch.bool, device=dev)
    rest[bad] = False
    assert torch.equal(dz[rest], clean[2][rest])


@pytest.mark.parametrize("T,V,dtype", SHAPES)
def test_no_advantage_means_no_term_whatever_the_ratio(lib, T, V, dtype):
    """Ratios beyond float32 (an old log-probability 100 to 300 below): 0 under
    advantage 0, as in float64, and the clipped product under a positive one."""
    z, a, old, adv, w, ref = batch(T, V, dtype, T + V + 1)
    rows = torch.arange(0, T, 5, device=dev)
    old[rows] = ref[rows] - 100 - 200 * torch.rand(len(rows), device=dev)
    adv[rows[::2]] = 0
    adv[rows[1::4]] = -0.0
    r = reference(z[:60], a[:60], old[:60], adv[:60], w[:60])
    loss, lp, dz = lib.policy_loss(z, a, old, adv, w)
    assert loss.isfinite().all() and dz.isfinite().all() and (dz[rows] == 0).all()
    check(lib.policy_loss(z[:60].contiguous(), a[:60], old[:60], adv[:60], w[:60]), r)
    adv[rows] = 0                       # without an upper clip the clipped ratio is as large
    loss, lp, dz = lib.policy_loss(z, a, old, adv, w, clip_high=float("inf"))
    assert loss.isfinite().all() and (dz[rows] == 0).all()
