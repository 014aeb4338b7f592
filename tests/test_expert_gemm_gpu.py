"""The experts' block-scaled products and their weights' gradient against
float64 products of the dequantized operands."""

import numpy as np
import pytest
import torch

from oracle import gemm as og
from tests.expert_reference import decoded, integer_operand, plan_of, routing

pytestmark = pytest.mark.gpu

dev = torch.device("cuda")
BF, F32 = torch.bfloat16, torch.float32
PAIRS = [("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e4m3", "e2m1"), ("e2m1", "e5m2"), ("e2m1", "e2m1")]


def make_plan(lib, tokens, top, experts, pattern, align, seed=0):
    e = routing(np.random.default_rng(seed), tokens, top, experts, pattern)
    return lib.expert_sort(torch.from_numpy(e).int().to(dev), experts, align), plan_of(e, experts, align)


def products(a, b, offsets, rows):
    """float64 C of stacked weights b [E][N][K]."""
    c = np.zeros((rows, b.shape[1]))
    for e in range(len(offsets) - 1):
        c[offsets[e]:offsets[e + 1]] = a[offsets[e]:offsets[e + 1]] @ b[e].T
    return c


def rounded(c, dtype):
    return torch.from_numpy(c).to(F32).to(dtype).double().numpy()


ROUTINGS = [(1, 1, 1, "even"), (1, 2, 8, "even"), (300, 2, 3, "even"), (700, 1, 5, "skewed"), (200, 2, 4, "one"),
            (50, 2, 3, "none"), (400, 2, 9, "dropped")]


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("fmt,b_fmt", PAIRS)
@pytest.mark.parametrize("align,n", [(128, 128), (128, 256), (256, 128), (256, 256), (256, 512)])
@pytest.mark.parametrize("tokens,top,experts,pattern", ROUTINGS)
def test_products_exactly(lib, tokens, top, experts, pattern, align, n, fmt, b_fmt, out):
    """Sums that are exact in float32 come out bit for bit: every expert, block,
    scale and zero tile is where it belongs."""
    p, want = make_plan(lib, tokens, top, experts, pattern, align)
    rng = np.random.default_rng(n)
    K = 256
    aq, as_ = integer_operand(rng, p.rows, K, fmt)
    bq, bs = integer_operand(rng, experts * n, K, b_fmt)
    c = lib.mx_expert_gemm(aq, as_, bq.view(experts, n, -1), bs, p, fmt, b_fmt, out)
    ref = products(decoded(aq, as_, fmt), decoded(bq, bs, b_fmt).reshape(experts, n, K), want[0], p.rows)
    assert c.dtype == out and np.array_equal(c.double().cpu().numpy(), rounded(ref, out))
    assert lib.last_device_status() == 0


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("fmt,b_fmt", PAIRS)
@pytest.mark.parametrize("align,n,k", [(128, 128, 256), (128, 640, 2304), (256, 256, 2048)])
@pytest.mark.parametrize("counts", [(1,), (0, 32), (31, 0, 1), (16, 1, 0, 8, 7), (33,), (0, 31, 2, 32), (129, 255, 64, 256, 1)])
def test_products_of_few_tokens(lib, counts, align, n, k, fmt, b_fmt, out):
    """Blocks with one token to a few, and what follows them: exact sums again,
    zeros behind the tokens."""
    experts = len(counts)
    e = torch.repeat_interleave(torch.arange(experts), torch.tensor(counts))
    p = lib.expert_sort(e[torch.randperm(len(e), generator=torch.Generator().manual_seed(4))].view(-1, 1).to(dev), experts, align)
    rng = np.random.default_rng(n + k)
    aq, as_ = integer_operand(rng, p.rows, k, fmt)
    aq[p.row_slot < 0] = 0
    bq, bs = integer_operand(rng, experts * n, k, b_fmt)
    ref = products(decoded(aq, as_, fmt), decoded(bq, bs, b_fmt).reshape(experts, n, k), p.offsets.tolist(), p.rows)
    for _ in range(2):
        c = lib.mx_expert_gemm(aq, as_, bq.view(experts, n, -1), bs, p, fmt, b_fmt, out)
        assert np.array_equal(c.double().cpu().numpy(), rounded(ref, out))
    assert lib.last_device_status() == 0


@pytest.mark.parametrize("fmt,b_fmt", PAIRS)
@pytest.mark.parametrize("align,n", [(128, 128), (256, 256)])
def test_products_with_experts_along_the_contraction(lib, align, n, fmt, b_fmt):
    experts, K = 5, 256
    p, want = make_plan(lib, 600, 1, experts, "skewed", align)
    rng = np.random.default_rng(7)
    aq, as_ = integer_operand(rng, p.rows, K, fmt)
    bq, bs = integer_operand(rng, n, experts * K, b_fmt)
    c = lib.mx_expert_gemm(aq, as_, bq, bs, p, fmt, b_fmt, F32)
    b = decoded(bq, bs, b_fmt).reshape(n, experts, K).transpose(1, 0, 2)
    assert np.array_equal(c.double().cpu().numpy(), products(decoded(aq, as_, fmt), b, want[0], p.rows))


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("fmt,b_fmt", PAIRS)
@pytest.mark.parametrize("align,n,k", [(128, 128, 128), (128, 256, 128), (256, 256, 256), (256, 512, 256), (256, 128, 384)])
@pytest.mark.parametrize("tokens,top,experts,pattern", ROUTINGS)
def test_weight_gradient_exactly(lib, tokens, top, experts, pattern, align, n, k, fmt, b_fmt, out):
    if fmt == b_fmt == "e2m1" and align != 256:
        return
    p, want = make_plan(lib, tokens, top, experts, pattern, align)
    rng = np.random.default_rng(n + k)
    aq, as_ = integer_operand(rng, n, p.rows, fmt)
    bq, bs = integer_operand(rng, k, p.rows, b_fmt)
    c = lib.mx_expert_wgrad(aq, as_, bq, bs, p, fmt, b_fmt, out)
    a, b, o = decoded(aq, as_, fmt), decoded(bq, bs, b_fmt), want[0]
    ref = np.stack([a[:, o[e]:o[e + 1]] @ b[:, o[e]:o[e + 1]].T for e in range(experts)])
    assert c.shape == (experts, n, k) and np.array_equal(c.double().cpu().numpy(), rounded(ref, out))
    assert lib.last_device_status() == 0


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("fmt,b_fmt", PAIRS)
@pytest.mark.parametrize("align,n", [(128, 2048), (128, 2176), (256, 1024), (256, 1152)])
def test_products_of_many_tiles_exactly(lib, align, n, fmt, b_fmt, out):
    """As many tiles as the wide tiles and the pairs take (of odd multiples of 128
    columns, too: the last tile reaches beyond C), an expert without rows among them."""
    experts, K = 5, 512
    e = np.minimum(routing(np.random.default_rng(2), 2500, 2, experts, "skewed") * 2, experts - 1)
    e[e == 3] = 4
    e[:30] = -1
    p = lib.expert_sort(torch.from_numpy(e).int().to(dev), experts, align)
    rng = np.random.default_rng(n)
    aq, as_ = integer_operand(rng, p.rows, K, fmt)
    bq, bs = integer_operand(rng, experts * n, K, b_fmt)
    ref = products(decoded(aq, as_, fmt), decoded(bq, bs, b_fmt).reshape(experts, n, K), p.offsets.tolist(), p.rows)
    for _ in range(2):
        c = lib.mx_expert_gemm(aq, as_, bq.view(experts, n, -1), bs, p, fmt, b_fmt, out)
        assert np.array_equal(c.double().cpu().numpy(), rounded(ref, out))
    assert lib.last_device_status() == 0


def blocks_of(rng, rows, k, fmt):
    """integer_operand's codes, scales and float64 values, of few blocks of 128
    rows that come again in a random order."""
    q, s = integer_operand(rng, 7 * 128, k, fmt)
    pick = torch.from_numpy(rng.integers(0, 7, size=rows // 128)).to(dev)
    v = decoded(q, s, fmt).reshape(7, 128, k)[pick.cpu().numpy()].reshape(rows, k)
    return q.view(7, 128, -1)[pick].view(rows, -1), s.view(7, -1)[pick].view(-1), v


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("fmt,b_fmt", PAIRS)
@pytest.mark.parametrize("align,n,steps", [(128, 1152, 8), (256, 1152, 7), (256, 1152, 16), (256, 640, 16), (256, 2176, 8)])
def test_products_of_odd_multiples_of_128_columns(lib, align, n, steps, fmt, b_fmt, out):
    """Contractions on both sides of where such products take 128 x 256 tiles and
    pairs, whose last tile reaches beyond C: exact sums, zeros behind the tokens."""
    experts = 5
    k = steps * (256 if fmt == b_fmt == "e2m1" else 128) * (2 if out == F32 else 1)
    rng = np.random.default_rng(n + steps)
    e = rng.integers(0, experts, size=(4300, 2))
    e[e == 3] = 4
    e[:300] = -1                                     # leaves blocks behind the last stretch
    p = lib.expert_sort(torch.from_numpy(e).int().to(dev), experts, align)
    off = p.offsets.tolist()
    assert off[experts] + 256 <= p.rows
    aq, as_, a = blocks_of(rng, p.rows, k, fmt)
    bq, bs, b = blocks_of(rng, experts * n, k, b_fmt)
    ref = products(a, b.reshape(experts, n, k), off, p.rows)
    for _ in range(2):
        c = lib.mx_expert_gemm(aq, as_, bq.view(experts, n, -1), bs, p, fmt, b_fmt, out)
        assert np.array_equal(c.double().cpu().numpy(), rounded(ref, out))
    assert lib.last_device_status() == 0


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("fmt,b_fmt", PAIRS)
@pytest.mark.parametrize("tokens,experts,n,k", [(700, 5, 1024, 2048), (700, 5, 1024, 2176), (1600, 2, 1536, 1792),
                                                  (1600, 2, 1536, 1920), (500, 6, 1152, 896)])
def test_weight_gradient_of_many_tiles_exactly(lib, tokens, experts, n, k, fmt, b_fmt, out):
    """Wide tiles, pairs (from 1536 rows an expert on) and small tiles, an expert without rows among them."""
    e = routing(np.random.default_rng(3), tokens, 2, experts, "even")
    if experts > 2:
        e[e == 1] = 0
    p = lib.expert_sort(torch.from_numpy(e).int().to(dev), experts, 256)
    rng = np.random.default_rng(n + k)
    aq, as_ = integer_operand(rng, n, p.rows, fmt)
    bq, bs = integer_operand(rng, k, p.rows, b_fmt)
    a, b, o = decoded(aq, as_, fmt), decoded(bq, bs, b_fmt), p.offsets.tolist()
    ref = np.stack([a[:, o[i]:o[i + 1]] @ b[:, o[i]:o[i + 1]].T for i in range(experts)])
    for _ in range(2):
        c = lib.mx_expert_wgrad(aq, as_, bq, bs, p, fmt, b_fmt, out)
        assert np.array_equal(c.double().cpu().numpy(), rounded(ref, out))
    assert lib.last_device_status() == 0


@pytest.mark.parametrize("align,n,k", [(128, 384, 1024), (256, 1024, 1152)])
def test_many_tiles_of_general_values(lib, align, n, k):
    """More tiles than teams (rings and accumulators go round), general values, within the products' gate of 2e-3."""
    experts = 11
    p, want = make_plan(lib, 3000, 2, experts, "skewed", align)
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(3000, k, device=dev, generator=g).to(BF)
    w = (0.02 * torch.randn(experts * n, k, device=dev, generator=g)).to(BF)
    dy = torch.randn(p.rows, n, device=dev, generator=g).to(BF)
    dy[p.row_slot < 0] = 0
    q, s, qT, sT = lib.mx_expert_gather(x, p, "e4m3", "dual", sf_layout="mma")
    wq, ws, wqT, wsT = lib.mx_quantize(w, "e4m3", "dual", sf_layout="mma")
    dq, ds, dqT, dsT = lib.mx_quantize(dy, "e5m2", "dual", sf_layout="mma")
    o = want[0]
    c = lib.mx_expert_gemm(q, s, wq.view(experts, n, k), ws, p)
    assert og.gate_error(c.double().cpu().numpy(), products(decoded(q, s, "e4m3"), decoded(wq, ws, "e4m3").reshape(experts, n, k), o, p.rows)) <= 2e-3
    # backward: the same weights' column copy, the experts along the contraction
    c = lib.mx_expert_gemm(dq, ds, wqT, wsT, p, "e5m2", "e4m3")
    b = decoded(wqT, wsT, "e4m3").reshape(k, experts, n).transpose(1, 0, 2)
    assert og.gate_error(c.double().cpu().numpy(), products(decoded(dq, ds, "e5m2"), b, o, p.rows)) <= 2e-3
    c = lib.mx_expert_wgrad(dqT, dsT, qT, sT, p, "e5m2", "e4m3")
    a, b = decoded(dqT, dsT, "e5m2"), decoded(qT, sT, "e4m3")
    ref = np.stack([a[:, o[e]:o[e + 1]] @ b[:, o[e]:o[e + 1]].T for e in range(experts)])
    assert og.gate_error(c.double().cpu().numpy(), ref, False) <= 2e-3
    # the same calls give the same bits
    assert torch.equal(c, lib.mx_expert_wgrad(dqT, dsT, qT, sT, p, "e5m2", "e4m3"))


def test_gradient_against_differences(lib):
    """C is linear in the weights: raising one weight by 1 changes <G, C> by the
    gradient's element, exactly where all sums are."""
    experts, n, k = 3, 128, 128
    p, want = make_plan(lib, 300, 1, experts, "even", 128)
    rng = np.random.default_rng(1)
    live = (p.row_slot >= 0)
    x = torch.from_numpy(rng.choice([0.0, 0.5, 1.0, -1.0], size=(p.rows, k))).to(BF).to(dev) * live[:, None]
    G = torch.from_numpy(rng.choice([0.0, 0.5, 1.0, -1.0], size=(p.rows, n))).to(BF).to(dev) * live[:, None]
    q, s, qT, sT = lib.mx_quantize(x, "e4m3", "dual", sf_layout="mma")
    gqT, gsT = lib.mx_quantize(G, "e4m3", "col", sf_layout="mma")[2:]
    dw = lib.mx_expert_wgrad(gqT, gsT, qT, sT, p)
    w = torch.from_numpy(rng.choice([0.0, 0.5, 1.0, -1.0], size=(experts, n, k))).to(BF).to(dev)

    def loss(weights):
        wq, ws, _, _ = lib.mx_quantize(weights.view(-1, k), "e4m3", "row", sf_layout="mma")
        return float((lib.mx_expert_gemm(q, s, wq.view(experts, n, k), ws, p, out_dtype=F32).double() * G.double()).sum())

    for _ in range(12):
        e, i, j = rng.integers(experts), rng.integers(n), rng.integers(k)
        up = w.clone()
        up[e, i, j] += 1
        assert loss(up) - loss(w) == float(dw[e, i, j])


def test_no_tokens(lib):
    p = lib.expert_sort(torch.empty(0, 2, dtype=torch.int32, device=dev), 3)
    z = lambda *shape: torch.zeros(*shape, dtype=torch.uint8, device=dev)
    assert lib.mx_expert_gemm(z(0, 128), z(0), z(3, 128, 128), z(3 * 128 * 4), p).shape == (0, 128)
    dw = lib.mx_expert_wgrad(z(128, 0), z(0), z(256, 0), z(0), p)
    assert dw.shape == (3, 128, 256) and not dw.any()


def test_a_wrong_plan_stays_within_bounds(lib):
    """Bounds and experts that no sort gives (a plan changed by hand): tiles stay within the operands."""
    p, _ = make_plan(lib, 300, 2, 4, "even", 128)
    rng = np.random.default_rng(2)
    aq, as_ = integer_operand(rng, p.rows, 128, "e4m3")
    bq, bs = integer_operand(rng, 4 * 128, 128, "e4m3")
    gq, gs = integer_operand(rng, 128, p.rows, "e4m3")
    few, _ = make_plan(lib, 16, 2, 4, "even", 128)
    fq, fs = integer_operand(rng, few.rows, 1024, "e4m3")
    wq, ws = integer_operand(rng, 4 * 128, 1024, "e4m3")
    off, block, big = p.offsets.clone(), p.block_expert.clone(), 2 ** 31 - 1
    for o, b in ((torch.full_like(off, big), torch.full_like(block, big)), (torch.full_like(off, -big), torch.full_like(block, -big)),
                 (off.flip(0), block.flip(0)), (off, torch.full_like(block, 1))):
        p.offsets.copy_(o)
        p.block_expert.copy_(b)
        lib.mx_expert_gemm(aq, as_, bq.view(4, 128, 128), bs, p)
        lib.mx_expert_wgrad(gq, gs, gq, gs, p)
        few.offsets.copy_(o)
        few.block_expert.copy_(b[:few.rows // 128])
        lib.mx_expert_gemm(fq, fs, wq.view(4, 128, 1024), ws, few)
    assert lib.last_device_status() == 0
