"""GPU tests of grad_norm and clip_grad_norm against the formula in float64.

Tolerances, u = 2^-24: a thread's batch adds at most 32 squares in a tree (five
additions and the squares' own rounding), float64 beyond; the norm is its
root, rounded once: 4 u.  The factor adds the sum, the quotient and the
product: 8 u on a float32 output, half an ulp more on bf16."""

import numpy as np
import pytest
import torch

from tests.rounding import half_ulp

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
dev = torch.device("cuda")
BF, F32 = torch.bfloat16, torch.float32


def d(t):
    return t.detach().cpu().double().numpy()


def norm_ref(gs):
    return float(np.sqrt(sum(float((d(g) ** 2).sum()) for g in gs)))


def grads(shapes, types, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(*s, generator=g) * scale).to(types[k % len(types)]).to(dev) for k, s in enumerate(shapes)]


def check(lib, gs, max_norm, out_types=None):
    want = norm_ref(gs)
    before = [d(g) for g in gs]
    n = lib.grad_norm(gs)
    assert n.shape == (1,) and n.dtype == F32 and abs(float(n) - want) <= 4 * U * want
    factor = min(1.0, max_norm / (want + 1e-6))
    outs = [torch.full_like(g, 7.0, dtype=out_types[k % len(out_types)]) for k, g in enumerate(gs)] if out_types else None
    n2 = lib.clip_grad_norm(gs, max_norm, out=outs)
    assert torch.equal(n, n2)
    for k, (g, b) in enumerate(zip(gs, before)):
        o = g if outs is None else outs[k]
        r = b * factor
        e = 8 * U * np.abs(r)
        assert (np.abs(d(o) - r) <= e + (half_ulp(BF, r, e) if o.dtype == BF else 1e-40)).all()
        if outs is not None:
            assert np.array_equal(d(g), b)


LISTS = [[(1,)], [(5,)], [(7,), (1,), (4096,)], [(2048,)], [(2049,)], [(3, 5, 7), (16385,)], [(1000, 1000)],
         [(129,), (129, 515), (515, 129), (1000, 129)], [(0,), (33,), (0, 4)], [(4000, 1003), (1,), (257, 255)]]


@pytest.mark.parametrize("shapes", LISTS)
@pytest.mark.parametrize("types", [[BF], [F32], [BF, F32]])
def test_lists_and_types(lib, shapes, types):
    for max_norm in (0.5, 1e9):
        check(lib, grads(shapes, types, len(shapes)), max_norm)
        check(lib, grads(shapes, types, len(shapes)), max_norm, [F32])
        check(lib, grads(shapes, types, len(shapes)), max_norm, [BF])


def test_many_tensors(lib):
    """More tensors than one launch's table holds, mixed sizes and types."""
    shapes = [(1 + (k * 37) % 700,) for k in range(1300)]
    check(lib, grads(shapes, [BF, F32, BF], 5), 1.0)
    check(lib, grads(shapes, [BF, F32, BF], 6), 1.0, [F32, BF])


def test_odd_bases(lib):
    """Tensors that start at any element of a buffer, outputs elsewhere."""
    for dt in (BF, F32):
        buf = grads([(50000,)], [dt], 7)[0]
        gs = [buf[1:1000], buf[1003:9001], buf[9002:9003], buf[10000:40001]]
        outbuf = torch.zeros(60000, dtype=F32, device=dev)
        outs = [outbuf[3:1002], outbuf[2000:9998], outbuf[1999:2000], outbuf[20001:50002]]
        want = norm_ref(gs)
        n = lib.clip_grad_norm(gs, 1.0, out=outs)
        assert abs(float(n) - want) <= 4 * U * want
        for g, o in zip(gs, outs):
            assert np.abs(d(o) - d(g) / (want + 1e-6)).max() <= 8 * U
        assert outbuf[0] == 0 and outbuf[1002] == 0 and outbuf[9998] == 0 and outbuf[50002] == 0


def test_transposed_gradients(lib):
    g = grads([(300, 200)], [F32], 8)[0]
    check(lib, [g.t(), grads([(64,)], [F32], 9)[0]], 1.0)
    o = torch.empty(300, 200, device=dev).t()
    lib.clip_grad_norm([g.t()], 1.0, out=[o])
    assert torch.equal(o, lib_scaled(lib, g).t())


def test_outputs_of_other_shapes(lib):
    """Stretches of a flat buffer take the elements in their order."""
    gs = grads([(12, 7), (5,), (3, 4, 2)], [F32], 14)
    flat = torch.zeros(200, device=dev)
    outs = [flat[:84], flat[96:101], flat[128:152]]
    lib.clip_grad_norm(gs, 0.5, out=outs)
    want = [lib_scaled_by(gs, g, 0.5) for g in gs]
    for o, w in zip(outs, want):
        assert (np.abs(d(o) - w) <= 8 * U * np.abs(w)).all()
    assert (flat[84:96] == 0).all() and (flat[152:] == 0).all()


def lib_scaled_by(gs, g, max_norm):
    return (d(g) * min(1.0, max_norm / (norm_ref(gs) + 1e-6))).reshape(-1)


def lib_scaled(lib, g):
    o = torch.empty_like(g)
    lib.clip_grad_norm([g], 1.0, out=[o])
    return o


def test_no_clipping_needed_leaves_the_bits(lib):
    gs = grads([(5000,), (33,)], [BF, F32], 10, 1e-3)
    before = [g.clone() for g in gs]
    lib.clip_grad_norm(gs, 10.0)
    assert all(torch.equal(a, b) for a, b in zip(gs, before))
    zeros = [torch.zeros(100, device=dev)]
    assert lib.clip_grad_norm(zeros, 1.0).item() == 0 and (zeros[0] == 0).all()


@pytest.mark.parametrize("scale", [1e25, 3e37, 1e-25, 1e-38])
def test_values_whose_squares_leave_float32(lib, scale):
    """The norm stays finite and exact where float32 squares overflow or vanish."""
    for n in (1, 7, 5000):
        g = torch.linspace(-1, 1, n, dtype=torch.float64) if n > 1 else torch.ones(1, dtype=torch.float64)
        g = (g * scale).float().to(dev)
        want = norm_ref([g])
        got = float(lib.grad_norm([g]))
        if want < 3.4e38:
            assert abs(got - want) <= 4 * U * want + 1e-45
        else:
            assert got == float("inf")


def test_mixed_magnitudes(lib):
    """Ordinary values beside values below 2^-50 and above 2^50 in one batch."""
    g = torch.full((4096,), 1e-20)
    g[::7] = 3.0
    h = torch.full((4096,), 1e-3)
    h[5] = 1e20
    for t in (g, h):
        want = norm_ref([t])
        assert abs(float(lib.grad_norm([t.to(dev)])) - want) <= 4 * U * want


def test_nonfinite_values(lib):
    g = grads([(3000,)], [F32], 11)[0]
    g[100] = float("inf")
    o = torch.empty_like(g)
    assert lib.clip_grad_norm([g], 1.0, out=[o]).item() == float("inf")
    assert o[100].isnan() and (o[:100] == 0).all()
    g[7] = float("nan")
    assert lib.clip_grad_norm([g], 1.0, out=[o]).isnan().all() and o.isnan().all()


def test_max_norm_zero(lib):
    gs = grads([(100,)], [F32], 12)
    lib.clip_grad_norm(gs, 0.0)
    assert (gs[0] == 0).all()


def test_same_bits_on_every_run_and_stream(lib):
    gs = grads([(129, 515)] * 20, [BF, F32], 13)
    first = lib.grad_norm(gs)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(10_000_000)
        again = lib.grad_norm(gs)
    s.synchronize()
    assert torch.equal(first, again)


def test_beyond_2_31_elements(lib):
    n = 2 ** 31 + 4099
    g = torch.ones(n, dtype=BF, device=dev)
    g[-1] = 3.0
    want = float(np.sqrt(n + 8.0))
    assert abs(float(lib.clip_grad_norm([g], 1024.0)) - want) <= 4 * U * want
    f = 1024.0 / (want + 1e-6)
    for at in (0, 2 ** 31 - 1, 2 ** 31, n - 2):
        assert abs(float(g[at]) - f) <= 2.0 ** -8 * f
    assert abs(float(g[-1]) - 3 * f) <= 2.0 ** -8 * 3 * f
