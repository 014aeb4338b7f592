"""policy_loss on long rows of many tokens: the ring of bulk-copied chunks, in
clusters of one, two, four and eight CTAs.  Several tokens to a cluster, rows
that start at every place of a 16-byte word, masks and undefined rows.  The
formula and the tolerances are those of the other policy-loss tests; a thread
of the ring adds at most 16 words and rescales its sum as often, which they
allow."""

import pytest
import torch

from tests.test_policy_loss_gpu import batch, check, d, reference

pytestmark = pytest.mark.gpu

dev = torch.device("cuda")
BF, F32 = torch.bfloat16, torch.float32
TYPES = [(BF, BF), (F32, F32), (F32, BF), (BF, F32)]


def tokens_for(V, zt, each=5):
    """About ``each`` tokens to a cluster of as many CTAs as hold a row (64 KiB each), two CTAs to an SM."""
    slabs = 1
    while V * (2 if zt == BF else 4) > 65536 * slabs:
        slabs *= 2
    assert slabs <= 8
    return each * 2 * torch.cuda.get_device_properties(0).multi_processor_count // slabs + 3


# per type of the logits: one to eight CTAs a row, even and odd widths, rows that end inside a chunk, a word, at a chunk's end
WIDTHS = {BF: [12296, 24577, 32752, 40003, 65537, 131071, 131072, 262000], F32: [16392, 20001, 32752, 50021, 65540, 131063]}


@pytest.mark.parametrize("zt,gt,V", [(zt, gt, V) for zt, gt in TYPES for V in WIDTHS[zt]])
def test_ring_shapes_and_types(lib, zt, gt, V):
    T = tokens_for(V, zt, 3 if V > 32768 else 2)
    z, a, old, adv, w, ref = batch(T, V, zt, T + V, masked=0.25)
    w[0] = w[-1] = 1.0 / T
    a[0], a[1], a[2] = 0, V - 1, V // 2
    lp = torch.log_softmax(z[:3].double(), 1)[torch.arange(3), a[:3]].float()
    old[:3] = lp - 0.02
    r = reference(z, a, old, adv, w, ref, beta=0.05, scale=3.0)
    out = lib.policy_loss(z, a, old, adv, w, ref_logp=ref, beta=0.05, grad_scale=3.0, grad_dtype=gt)
    check(out, r)
    assert (out[2][w == 0] == 0).all() and (out[1][w == 0] == 0).all()
    bare = lib.policy_loss(z, a, old, adv, w, ref_logp=ref, beta=0.05, grad=False)
    assert bare[2] is None
    check(bare, reference(z, a, old, adv, w, ref, beta=0.05))
    if zt == gt:            # the same kernel (another type of gradient may split a row otherwise)
        assert torch.equal(bare[0], out[0]) and torch.equal(bare[1], out[1])


@pytest.mark.parametrize("zt,V,pad,shift", [(BF, 12297, 7, 0), (BF, 12296, 8, 8), (F32, 16393, 3, 0), (F32, 20000, 4, 4),
                                            (BF, 40003, 5, 0)])
def test_ring_strided_logits_without_gradient(lib, zt, V, pad, shift):
    """Slices of padded logits; with no gradient to be in step with, rows may start anywhere."""
    T = tokens_for(V, zt, 2)
    z, a, old, adv, w, ref = batch(T, V + pad, zt, T, masked=0.1)
    z = z[:, shift:shift + V]
    a = a % V
    old = torch.log_softmax(z.double(), 1)[torch.arange(T), a].float() - 0.03
    loss, lp, _ = lib.policy_loss(z, a.int(), old, adv, w, grad=False)
    rl, rp, _, el, ep, _ = reference(z, a, old, adv, w)
    assert abs(float(loss) - rl) <= el + 2.0 ** -24 * abs(rl)
    assert (abs(d(lp) - rp) <= ep).all()


@pytest.mark.parametrize("zt,V", [(BF, 12296), (F32, 16393), (BF, 65537), (F32, 50021)])
@pytest.mark.parametrize("share", [0.5, 0.97])
def test_ring_masked_tokens_are_not_looked_at(lib, zt, V, share):
    """Weight 0: NaN logits, any target, NaN statistics; the other rows keep their bits."""
    T = tokens_for(V, zt, 4)
    z, a, old, adv, w, ref = batch(T, V, zt, 31, masked=share)
    w[-1] = 1.0 / T
    clean = lib.policy_loss(z, a, old, adv, w, ref_logp=ref, beta=0.1)
    off = w == 0
    z[off] = float("nan")
    a[off] = -2 ** 40
    for t in (old, adv, ref):
        t[off] = float("nan")
    out = lib.policy_loss(z, a, old, adv, w, ref_logp=ref, beta=0.1)
    for x, y in zip(out, clean):
        assert torch.equal(x, y)
    assert (out[2][off] == 0).all() and (out[1][off] == 0).all()
    loss, lp, dz = lib.policy_loss(z, a, old, adv, torch.zeros_like(w), ref_logp=ref, beta=0.1)
    assert loss.item() == 0 and (lp == 0).all() and (dz == 0).all()


@pytest.mark.parametrize("zt,V", [(BF, 12297), (F32, 16392), (BF, 131071), (F32, 65537)])
def test_ring_masked_vocabulary(lib, zt, V):
    """Logits of -inf and of the type's lowest value: whole chunks, whole CTAs and the ragged ends of them."""
    T = tokens_for(V, zt, 3)
    z, a, old, adv, w, ref = batch(T, V, zt, 33)
    low = torch.finfo(zt).min
    a = torch.arange(T, device=dev) % 5
    z[0::5, 1:] = float("-inf")
    z[1::5, 10:] = low
    z[2::5, 10:V - 3] = float("-inf")
    z[3::5, 5:] = float("-inf")
    z[4::5] = float("-inf")
    z[4::5, 4] = low
    z[4::5, V - 1] = low
    old = torch.log_softmax(z.double(), 1)[torch.arange(T), a].float() - 0.02
    out = lib.policy_loss(z, a, old, adv, w)
    zz = torch.where(z == float("-inf"), torch.tensor(low, dtype=zt, device=dev), z)
    zz[4::5] = -1e4                                    # two equal logits, the rest far below
    zz[4::5, 4] = zz[4::5, V - 1] = 0.0
    check(out, reference(zz, a, old, adv, w))
    assert (out[2][0::5, 1:] == 0).all() and (out[2][4::5, 5:V - 1] == 0).all()


@pytest.mark.parametrize("zt,V", [(BF, 12296), (F32, 16393), (F32, 50021)])
def test_ring_undefined_rows_stay_alone(lib, zt, V):
    """No finite logit, a NaN logit (in the first and last word, in the middle), +inf, targets outside the vocabulary."""
    T = tokens_for(V, zt, 3)
    z, a, old, adv, w, ref = batch(T, V, zt, 34)
    clean = lib.policy_loss(z, a, old, adv, w)
    bad = [1, 4, 5, T // 2, T // 2 + 1, T - 3, T - 1]
    z[bad[0]] = float("-inf")
    z[bad[1], 0] = z[bad[2], V - 1] = z[bad[3], V // 2] = float("nan")
    z[bad[4], 9] = float("inf")
    a[bad[5]], a[bad[6]] = V, -1
    loss, lp, dz = lib.policy_loss(z, a, old, adv, w)
    assert loss.isnan().all() and lp[bad].isnan().all() and dz[bad].isnan().all()
    keep = torch.ones(T, dtype=torch.bool, device=dev)
    keep[bad] = False
    assert torch.equal(lp[keep], clean[1][keep]) and torch.equal(dz[keep], clean[2][keep])


def test_ring_clipping_on_each_side(lib):
    V = 16392
    T = tokens_for(V, F32, 3) // 6 * 6
    z, a, old, adv, w, ref = batch(T, V, F32, 35)
    lp = torch.log_softmax(z.double(), 1)[torch.arange(T), a].float()
    old = lp - torch.tensor([0.5, 0.5, 1.0, 1.0, 2.0, 2.0], device=dev).repeat(T // 6).log()
    adv = torch.tensor([1.0, -1.0], device=dev).repeat(T // 2)
    out = lib.policy_loss(z, a, old, adv, w, clip_low=0.1, clip_high=0.3)
    check(out, reference(z, a, old, adv, w, lo=0.1, hi=0.3))
    assert (out[2].abs().sum(1) > 0).tolist() == [True, False, True, True, False, True] * (T // 6)


@pytest.mark.parametrize("zt,V", [(BF, 131072), (F32, 50021)])
def test_ring_same_bits_on_every_run_and_stream(lib, zt, V):
    z, a, old, adv, w, ref = batch(tokens_for(V, zt, 4), V, zt, 36, masked=0.3)
    first = lib.policy_loss(z, a, old, adv, w, ref_logp=ref, beta=0.1)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s):
            out = lib.policy_loss(z, a, old, adv, w, ref_logp=ref, beta=0.1)
        s.synchronize()
        for x, y in zip(out, first):
            assert torch.equal(x, y)
