"""Dropout against the oracle's generator and float64 arithmetic."""

import numpy as np
import pytest
import torch

from oracle import philox
from tests.rounding import half_ulp

pytestmark = pytest.mark.gpu

dev = torch.device("cuda")
BF, F32 = torch.bfloat16, torch.float32


def kept(rows, cols, p, seed, offset):
    i = np.arange(rows * cols, dtype=np.uint64) + np.uint64((4 * offset) % 2 ** 64)
    draw = philox.sr_draw4(seed, i).reshape(rows, cols)
    return draw.astype(np.float64) >= min(np.rint(p * 2.0 ** 32), 2.0 ** 32 - 1)


def check(lib, x, p, seed, offset, res=None, y=None):
    rows, cols = x.shape
    y = lib.dropout(x, p, seed, offset, residual=res) if y is None else y
    keep = kept(rows, cols, p, seed, offset)
    term = np.where(keep, x.double().cpu().numpy(), 0.0) / (1.0 - p)
    ref = term if res is None else term + res.double().cpu().numpy()
    # the factor and the product are off by half a step of the term each, the float32 sum by one of itself
    tol = 2.0 ** -23 * np.abs(term) * (1 + 1e-6)
    if res is not None:
        tol = tol + 2.0 ** -24 * (np.abs(ref) + tol)
    got = y.double().cpu().numpy()
    assert y.dtype == x.dtype and np.all(np.abs(got - ref) <= tol + half_ulp(x.dtype, ref, tol) * (ref != 0))
    if res is None:
        assert np.array_equal(got != 0, keep & (x.double().cpu().numpy() != 0))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 0.999])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 3), (1, 8), (3, 5), (7, 129), (64, 256), (333, 1021), (1, 40000)])
def test_dropout(lib, rows, cols, p, dtype):
    x = torch.randn(rows, cols, device=dev).to(dtype)
    res = torch.randn(rows, cols, device=dev).to(dtype)
    check(lib, x, p, 0x123456789ABCDEF, 77)
    check(lib, x, p, 2 ** 64 - 1, 0, res)


@pytest.mark.parametrize("res", [False, True])
def test_long_tensors(lib, res):
    """Four vectors to a thread, and a last element that fills none."""
    x = torch.randn(4099, 4101, device=dev).to(BF)
    check(lib, x, 0.2, 99, 11, torch.randn_like(x) if res else None)


@pytest.mark.parametrize("offset", [0, 2 ** 32 - 3, 2 ** 40 + 5, 2 ** 62 - 100])
def test_counters_pass_32_bits(lib, offset):
    check(lib, torch.randn(9, 40, device=dev), 0.3, 5, offset)
    check(lib, torch.randn(9, 41, device=dev), 0.3, 5, offset)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shift,pad", [(0, 8), (1, 0), (1, 3), (0, 1)])
def test_strided_and_shifted(lib, dtype, shift, pad):
    """The draw goes by the element's index, not by where it lies."""
    store = torch.randn(2, 20 * (128 + pad) + shift, device=dev).to(dtype)
    x, res = (s[shift:].view(20, 128 + pad)[:, :128] for s in store)
    want = lib.dropout(x.contiguous(), 0.25, 9, 3, residual=res.contiguous())
    assert torch.equal(lib.dropout(x, 0.25, 9, 3, residual=res), want)
    assert torch.equal(lib.dropout(x, 0.25, 9, 3, residual=res.contiguous()), want)
    check(lib, x, 0.25, 9, 3, res)


def test_what_is_dropped_is_not_looked_at(lib):
    keep = torch.from_numpy(kept(64, 96, 0.4, 3, 0)).to(dev)
    x = torch.where(keep, torch.randn(64, 96, device=dev), torch.tensor(float("nan"), device=dev))
    x[~keep] = torch.where(torch.arange(int((~keep).sum()), device=dev) % 2 == 0, float("inf"), float("nan"))
    y = lib.dropout(x, 0.4, 3)
    assert bool(torch.isfinite(y).all()) and not bool(y[~keep].any())


def test_backward_has_the_same_mask_and_differences_agree(lib):
    x, dy = torch.randn(2, 50, 70, device=dev)
    dx = lib.dropout(dy, 0.3, 21, 4)
    keep = torch.from_numpy(kept(50, 70, 0.3, 21, 4)).to(dev)
    assert torch.equal(dx != 0, keep & (dy != 0))
    up, down = lib.dropout(x + 1, 0.3, 21, 4), lib.dropout(x - 1, 0.3, 21, 4)
    slope = (up.double() - down.double()) / 2 * dy.double()
    # (x + 1) - (x - 1) is off by a step of each; the product by one more
    tol = 2.0 ** -22 * (x.abs() + 1).double() / 0.7 * dy.abs().double()
    assert bool(((slope - dx.double()).abs() <= tol + 2.0 ** -22 * dx.abs().double()).all())


def test_offset_on_the_device_and_in_a_graph(lib):
    x = torch.randn(40, 100, device=dev).to(BF)
    at = torch.tensor([5], device=dev)
    assert torch.equal(lib.dropout(x, 0.5, 1, at), lib.dropout(x, 0.5, 1, 5))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = lib.dropout(x, 0.5, 1, at)
        at += 1000
    for k in range(3):
        g.replay()
        check(lib, x, 0.5, 1, 5 + 1000 * k, y=y)


def test_share_of_kept_elements(lib):
    """2^22 draws: the share lies within 6 standard deviations of 1 - p."""
    x = torch.ones(2048, 2048, device=dev)
    for p in (0.05, 0.5):
        share = float((lib.dropout(x, p, 1234) != 0).double().mean())
        assert abs(share - (1 - p)) <= 6 * (p * (1 - p) / 2 ** 22) ** 0.5


def test_no_rows(lib):
    assert lib.dropout(torch.empty(0, 8, device=dev), 0.1, 0).shape == (0, 8)
