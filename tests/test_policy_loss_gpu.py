"""GPU tests of policy_loss against its formula in float64.

Tolerances, u = 2^-24: the sum of a row's exponentials has at most 30
roundings in its tree, each exponential the hardware's 2 ulp and the rounding
of its argument, u |z_v - max| twice, whose mean under the softmax is at most
log(vocab) + 1; the row's log-probability adds the roundings of its own
magnitude.  The rounding to the gradient's type adds half an ulp."""

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


def reference(z, a, old, adv, w, ref=None, lo=0.2, hi=0.2, beta=0.0, scale=1.0):
    """loss, logp, dlogits and their bounds."""
    z, old, adv, w = d(z), d(old), d(adv), d(w)
    a = a.cpu().numpy()
    T, V = z.shape
    live = w != 0
    loss, e_loss = 0.0, 0.0
    lp, e_lp = np.zeros(T), np.zeros(T)
    dz, e_dz = np.zeros((T, V)), np.zeros((T, V))
    for t in np.nonzero(live)[0]:
        top = z[t].max()
        ex = np.exp(z[t] - top)
        total = ex.sum()
        x = (z[t, a[t]] - top) - np.log(total)
        e = U * (60 + 4 * np.log(V) + 2 * abs(z[t, a[t]] - top) + 2 * abs(x))
        lp[t], e_lp[t] = x, e
        r = np.exp(x - old[t])
        e_r = r * (e + U * abs(x - old[t]) + 4 * U)
        c = min(max(r, 1 - lo), 1 + hi)
        free = r * adv[t] <= c * adv[t]
        l = -min(r * adv[t], c * adv[t])
        e_l = abs(adv[t]) * (e_r + 4 * U * max(r, c))
        s = -adv[t] * r if free else 0.0
        e_s = abs(adv[t]) * (e_r + 2 * U * r) if free else 0.0
        if beta:
            k = d(ref)[t] - x
            e_k = e + U * abs(k)
            l += beta * (np.expm1(k) - k)
            e_l += beta * (e_k * (abs(np.expm1(k)) + np.exp(k)) + 8 * U * (abs(np.expm1(k)) + abs(k)))
            s -= beta * np.expm1(k)
            e_s += beta * (np.exp(k) * e_k + 6 * U * abs(np.expm1(k)))
        loss += w[t] * l
        e_loss += abs(w[t]) * (e_l + 2 * U * abs(l))
        coef = scale * w[t] * s
        e_c = abs(scale * w[t]) * (e_s + 4 * U * abs(s))
        p = ex / total
        hot = np.zeros(V)
        hot[a[t]] = 1.0
        dz[t] = coef * (hot - p)
        e_p = p * (e + U * (12 + 4 * np.abs(z[t] - top)))
        e_dz[t] = abs(coef) * (e_p + 2 * U * (hot + p)) + e_c * np.abs(hot - p) + 1e-38
    return loss, lp, dz, e_loss, e_lp, e_dz


def batch(T, V, zt, seed, masked=0.0, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(T, V, generator=g) * spread
    a = torch.randint(V, (T,), generator=g)
    z[torch.arange(T), a] += 3.0
    z = z.to(zt)
    lp = torch.log_softmax(z.double(), 1)[torch.arange(T), a].float()
    drift = (torch.randn(T, generator=g) * 15).round() * 0.01
    adv = torch.randn(T, generator=g)
    w = (torch.rand(T, generator=g) >= masked).float() * (0.5 + torch.rand(T, generator=g)) / T
    ref = lp + 0.3 * torch.randn(T, generator=g)
    return [t.to(dev) for t in (z, a, lp - drift, adv, w, ref)]


def check(out, ref):
    loss, lp, dz = out
    rl, rp, rz, el, ep, ez = ref
    assert loss.shape == (1,) and loss.dtype == F32
    assert abs(float(loss) - rl) <= el + U * abs(rl)
    assert (np.abs(d(lp) - rp) <= ep).all()
    if dz is not None:
        assert (np.abs(d(dz) - rz) <= ez + half_ulp(dz.dtype, rz, ez)).all()


@pytest.mark.parametrize("T,V", [(1, 1), (3, 2), (1, 7), (2, 8), (5, 33), (4, 511), (3, 4096), (2, 4099), (300, 64),
                                 (7, 16384), (2, 16391), (400, 1000), (2, 32001), (1, 50021), (1, 131072), (1, 131071),
                                 (1, 131080), (2, 150001)])
@pytest.mark.parametrize("zt,gt", [(BF, BF), (F32, F32), (F32, BF), (BF, F32)])
def test_shapes_and_types(lib, T, V, zt, gt):
    z, a, old, adv, w, ref = batch(T, V, zt, T + V)
    for beta in (0.0, 0.05):
        r = reference(z, a, old, adv, w, ref, beta=beta, scale=3.0)
        check(lib.policy_loss(z, a, old, adv, w, ref_logp=ref, beta=beta, grad_scale=3.0, grad_dtype=gt), r)
    assert lib.policy_loss(z, a, old, adv, w, grad=False)[2] is None


@pytest.mark.parametrize("V", [1000, 1003, 16385])
@pytest.mark.parametrize("shift", [0, 1, 4, 8])
def test_strided_logits_and_int32_targets(lib, V, shift):
    """A slice of padded logits: rows that start anywhere, and a gradient whose
    rows start elsewhere within their 16 bytes."""
    for zt, gt in ((BF, BF), (F32, BF)):
        z, a, old, adv, w, ref = batch(6, V + 21, zt, V + shift)
        z = z[:, shift:shift + V]
        a = a % V
        lp = torch.log_softmax(z.double(), 1)[torch.arange(6), a].float()
        old = lp - 0.03
        r = reference(z, a, old, adv, w)
        check(lib.policy_loss(z, a.int(), old, adv, w, grad_dtype=gt), r)


@pytest.mark.parametrize("T,V", [(9800, 100), (3700, 1001), (1900, 5001), (1200, 7000), (200, 5000), (200, 8193),
                                 (920, 9001), (700, 12290)])
@pytest.mark.parametrize("zt,gt", [(BF, BF), (F32, BF)])
@pytest.mark.parametrize("pad", [0, 3])
def test_many_tokens(lib, T, V, zt, gt, pad):
    """Enough tokens that a row brings a later one near, masked ones among
    them, up to the last row of the matrix; padded rows of any alignment."""
    z, a, old, adv, w, ref = batch(T, V, zt, T + V, masked=0.8)
    w[-1] = w[0] = 1.0 / T
    if pad:
        wide = torch.full((T, V + pad), 7.0, device=dev, dtype=zt)
        wide[:, :V] = z
        z = wide[:, :V]
    r = reference(z, a, old, adv, w, ref)
    check(lib.policy_loss(z, a, old, adv, w, grad_dtype=gt), r)


def test_clipping_on_each_side(lib):
    """Ratios 0.5, 1, 2 with advantages of both signs, asymmetric clip: the
    slope is zero exactly where the clipped product is the smaller."""
    V = 100
    z = torch.randn(6, V, generator=torch.Generator().manual_seed(3)).to(dev)
    a = torch.arange(6, device=dev)
    lp = torch.log_softmax(z, 1)[a, a]
    old = lp - torch.tensor([0.5, 0.5, 1.0, 1.0, 2.0, 2.0], device=dev).log()
    adv = torch.tensor([1.0, -1.0] * 3, device=dev)
    w = torch.ones(6, device=dev)
    out = lib.policy_loss(z, a, old, adv, w, clip_low=0.1, clip_high=0.3)
    check(out, reference(z, a, old, adv, w, lo=0.1, hi=0.3))
    active = out[2].abs().sum(1) > 0
    assert active.tolist() == [True, False, True, True, False, True]


def test_masked_tokens_are_not_looked_at(lib):
    """Weight 0: NaN logits, any target, NaN statistics; logp and gradient 0 and the other rows unchanged."""
    for T, V in ((9, 5000), (5, 40001)):
        z, a, old, adv, w, ref = batch(T, V, F32, 21)
        w = torch.full_like(w, 1.0 / T)
        w[[1, T - 1]] = 0
        clean = lib.policy_loss(z, a, old, adv, w, ref_logp=ref, beta=0.1)
        z[1], z[T - 1] = float("nan"), float("-inf")
        a[1], a[T - 1] = -100, 2 ** 40
        for t in (old, adv, ref):
            t[1], t[T - 1] = float("nan"), float("inf")
        out = lib.policy_loss(z, a, old, adv, w, ref_logp=ref, beta=0.1)
        for x, y in zip(out, clean):
            assert torch.equal(x, y)
        assert (out[2][[1, T - 1]] == 0).all() and out[1][1] == 0


def test_every_token_masked(lib):
    z, a, old, adv, w, ref = batch(4, 777, BF, 22)
    loss, lp, dz = lib.policy_loss(z, a, old, adv, torch.zeros_like(w))
    assert loss.item() == 0 and (lp == 0).all() and (dz == 0).all()


def test_no_tokens(lib):
    e = torch.empty(0, device=dev)
    loss, lp, dz = lib.policy_loss(torch.empty(0, 50, device=dev), e.long(), e, e, e)
    assert loss.item() == 0 and lp.numel() == 0 and dz.shape == (0, 50)


def test_masked_vocabulary(lib):
    """Logits of -inf and of the type's lowest value are tokens of probability
    0; rows that have most of them (whole warps, whole CTAs) stay exact."""
    for zt in (BF, F32):
        for V in (900, 70001):
            z, a, old, adv, w, ref = batch(4, V, zt, 23)
            z[0, 10:] = float("-inf")
            z[1, 10:] = torch.finfo(zt).min
            z[2, :-3] = float("-inf")
            z[3, 1:] = float("-inf")
            a = torch.tensor([2, 9, V - 2, 0], device=dev)
            lp = torch.log_softmax(z.double(), 1)[torch.arange(4), a].float()
            out = lib.policy_loss(z, a, lp - 0.02, adv, w)
            zz = torch.where(z == float("-inf"), torch.tensor(torch.finfo(zt).min, dtype=zt, device=dev), z)
            check(out, reference(zz, a, lp - 0.02, adv, w))
            assert (out[2][0, 10:] == 0).all() and (out[2][2, :-3] == 0).all()


def test_undefined_rows_give_nan_and_stay_alone(lib):
    """No finite logit, a NaN logit, +inf, a target outside the vocabulary."""
    z, a, old, adv, w, ref = batch(8, 3000, F32, 24)
    clean = lib.policy_loss(z, a, old, adv, w)
    z[1] = float("-inf")
    z[3, 77] = float("nan")
    z[5, 9] = float("inf")
    a[7] = 3000
    loss, lp, dz = lib.policy_loss(z, a, old, adv, w)
    assert loss.isnan().all()
    for t in (1, 3, 5, 7):
        assert lp[t].isnan() and dz[t].isnan().all()
    for t in (0, 2, 4, 6):
        assert lp[t] == clean[1][t] and torch.equal(dz[t], clean[2][t])


def test_large_logits(lib):
    """Logits around 3e4: the maximum leaves before the exponential."""
    z, a, old, adv, w, ref = batch(3, 2000, F32, 25)
    z += 3.0e4
    lp = torch.log_softmax(z.double(), 1)[torch.arange(3), a].float()
    check(lib.policy_loss(z, a, lp - 0.01, adv, w), reference(z, a, lp - 0.01, adv, w))


def test_gradient_against_differences(lib):
    """Central differences of the float64 loss, step 1e-5 (truncation of the order 1e-10)."""
    T, V = 3, 40
    z, a, old, adv, w, ref = batch(T, V, F32, 26)
    _, _, dz = lib.policy_loss(z, a, old, adv, w, ref_logp=ref, beta=0.2)

    def f(zz):
        return reference(torch.from_numpy(zz), a, old, adv, w, ref, beta=0.2)[0]

    Z = d(z)
    for t, v in [(0, 0), (1, 17), (2, 39), (0, int(a[0])), (1, int(a[1])), (2, int(a[2]))]:
        e = np.zeros_like(Z)
        e[t, v] = 1e-5
        assert abs((f(Z + e) - f(Z - e)) / 2e-5 - d(dz)[t, v]) < 1e-6


def test_same_bits_on_every_run_and_stream(lib):
    z, a, old, adv, w, ref = batch(700, 3001, BF, 27, masked=0.3)
    first = lib.policy_loss(z, a, old, adv, w, ref_logp=ref, beta=0.1)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s):
            out = lib.policy_loss(z, a, old, adv, w, ref_logp=ref, beta=0.1)
        s.synchronize()
        for x, y in zip(out, first):
            assert torch.equal(x, y)


def test_beyond_2_31_elements(lib):
    T, V = 16400, 131072
    z = torch.empty(T, V, dtype=BF, device=dev)
    g = torch.Generator(device="cuda").manual_seed(2)
    for i in range(0, T, 1024):
        z[i:i + 1024].normal_(generator=g)
    a = torch.randint(V, (T,), device=dev, generator=g)
    w = torch.full((T,), 1.0 / T, device=dev)
    adv = torch.randn(T, device=dev, generator=g)
    old = torch.full((T,), -12.3, device=dev)
    loss, lp, dz = lib.policy_loss(z, a, old, adv, w)
    pick = [0, 8191, 16383, 16384, T - 1]
    _, rp, rz, _, ep, ez = reference(z[pick], a[pick], old[pick], adv[pick], w[pick])
    assert (np.abs(d(lp[pick]) - rp) <= ep).all()
    assert (np.abs(d(dz[pick]) - rz) <= ez + half_ulp(BF, rz, ez)).all()
