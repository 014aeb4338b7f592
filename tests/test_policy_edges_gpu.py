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
