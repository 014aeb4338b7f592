"""The training-step operators together, as examples/policy_step.py uses them:
the step's gradients against a float32 autograd model of the same layer, and
the task learned."""

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("policy_step", os.path.join(ROOT, "examples", "policy_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_gradients_match_float32_autograd(lib, example):
    """MXFP8 operands carry 3 (E4M3) and 2 (E5M2) mantissa bits: a rounding is
    at most 2^-4 and 2^-3 relative, so a gradient of two such factors is off by
    at most about 0.19 of its terms' magnitudes and, its errors being
    independent, by far less in the norm: 0.1."""
    T, D, V = 256, 256, 512
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(T, D, device="cuda", generator=g)
    targets = torch.randint(V, (T,), device="cuda", generator=g)
    adv = torch.randn(T, device="cuda", generator=g)
    w = torch.full((T,), 1.0 / T, device="cuda")
    layer = example.OutputLayer(D, V, 1)
    params = [p.clone().requires_grad_(True) for p in layer.params]
    xr = x.clone().requires_grad_(True)
    h = torch.nn.functional.layer_norm(xr, (D,), params[0], params[1])
    lp = torch.log_softmax(h @ params[2].t(), 1)[torch.arange(T), targets]
    (-(w * adv * torch.exp(lp - lp.detach())).sum()).backward()
    loss, logp, norm, dx = layer.step(x, targets, None, None, adv, w, lr=0.0, max_norm=1e9, beta=0.0)
    assert (logp - lp.detach()).abs().max() < 0.5
    for got, want in zip(layer.grads + [dx], [p.grad for p in params] + [xr.grad]):
        assert (got - want).norm() <= 0.1 * want.norm()
    total = torch.stack([g.norm() for g in layer.grads]).norm()
    assert abs(float(norm) / float(total) - 1) < 1e-5


def test_the_task_is_learned(lib, example):
    """Good tokens become likelier, bad ones less likely, in step with the loss."""
    t = example.train(12)
    assert t.isfinite().all()
    assert t[-1, 0] > t[0, 0] + 0.5 and t[-1, 1] < t[0, 1] - 0.5
    assert lib.last_device_status() == 0
