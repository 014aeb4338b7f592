"""Tokens sorted by expert, gathered (plain and to MX), and combined again, with
gradients, against plain 64-bit forms."""

import numpy as np
import pytest
import torch

from tests.expert_reference import plan_of, routing
from tests.rounding import half_ulp

pytestmark = pytest.mark.gpu

dev = torch.device("cuda")
BF, F32 = torch.bfloat16, torch.float32
PATTERNS = ["even", "skewed", "one", "none", "dropped"]


def make_plan(lib, rng, tokens, top, experts, pattern="even", align=128, dtype=torch.int32):
    e = routing(rng, tokens, top, experts, pattern)
    return lib.expert_sort(torch.from_numpy(e).to(dtype).to(dev), experts, align), plan_of(e, experts, align)


def np64(t):
    return t.double().cpu().numpy()


# ------------------------------------------------------------------ sort
@pytest.mark.parametrize("pattern", PATTERNS)
@pytest.mark.parametrize("tokens,top,experts", [(1, 1, 1), (1, 8, 64), (3, 2, 7), (100, 3, 5), (515, 2, 16), (2048, 1, 1024),
                                                (2049, 1, 2), (3000, 2, 9), (5000, 2, 12), (12289, 1, 40), (4097, 5, 33), (5000, 8, 1000), (8192, 4, 64), (8192, 8, 64), (32769, 1, 20), (300000, 1, 128)])
def test_sort(lib, tokens, top, experts, pattern):
    rng = np.random.default_rng(tokens + experts)
    for align, dtype in ((128, torch.int32), (256, torch.int64)):
        got, want = make_plan(lib, rng, tokens, top, experts, pattern, align, dtype)
        for name, w in zip(("offsets", "counts", "slot_row", "row_slot", "block_expert"), want):
            t = getattr(got, name)
            assert t.dtype == torch.int32 and np.array_equal(t.cpu().numpy(), w), name
        assert (got.tokens, got.top, got.experts, got.rows, got.align) == (tokens, top, experts, len(want[3]), align)


def test_alignment_by_default(lib):
    """Longer blocks from 256 slots an expert on."""
    for tokens, want in ((1, 128), (511, 128), (512, 256), (4000, 256)):
        assert lib.expert_sort(torch.zeros(tokens, 1, dtype=torch.int32, device=dev), 2).align == want


def test_sort_of_values_beyond_32_bits(lib):
    e = torch.tensor([[1, 1 + 2 ** 32], [2 ** 63 - 1, -(2 ** 63)], [2 ** 33, 0]], device=dev)
    p = lib.expert_sort(e, 4)
    assert p.slot_row.tolist() == [[128, -1], [-1, -1], [-1, 0]]
    assert p.counts.tolist() == [1, 1, 0, 0] and p.offsets.tolist() == [0, 128, 256, 256, 256]


def test_sort_of_no_tokens(lib):
    p = lib.expert_sort(torch.empty(0, 2, dtype=torch.int32, device=dev), 5)
    assert p.rows == 0 and p.offsets.tolist() == [0] * 6 and p.counts.tolist() == [0] * 5
    assert lib.expert_gather(torch.empty(0, 64, device=dev), p).shape == (0, 64)
    assert [None if t is None else t.numel() for t in lib.mx_expert_gather(torch.empty(0, 64, dtype=BF, device=dev), p)] == \
        [0, 0, None, None]
    assert lib.expert_combine(torch.empty(0, 64, device=dev), p).shape == (0, 64)
    d, w = lib.expert_combine_backward(torch.empty(0, 64, device=dev), torch.empty(0, 64, device=dev), p,
                                       torch.empty(0, 2, device=dev))
    assert d.shape == (0, 64) and w.shape == (0, 2)


# ------------------------------------------------------------------ gather
@pytest.mark.parametrize("pattern", ["even", "dropped", "none"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("tokens,top,experts,cols", [(1, 1, 1, 1), (1, 8, 64, 4096), (5, 2, 3, 7), (33, 3, 5, 1021),
                                                     (130, 2, 4, 1024), (257, 1, 300, 520), (70, 4, 8, 5000)])
def test_gather(lib, tokens, top, experts, cols, dtype, pattern):
    rng = np.random.default_rng(cols)
    p, want = make_plan(lib, rng, tokens, top, experts, pattern)
    bits = torch.int16 if dtype == BF else torch.int32
    info = torch.iinfo(bits)
    # any bit patterns, NaN payloads among them
    x = torch.from_numpy(rng.integers(info.min, info.max, size=(tokens, cols), dtype=np.int64)).to(bits).to(dev)
    got = lib.expert_gather(x.view(dtype), p).view(bits).cpu().numpy()
    row = want[3]
    ref = np.where((row >= 0)[:, None], x.cpu().numpy()[np.maximum(row, 0) // top], 0)
    assert np.array_equal(got, ref)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shift,pad", [(0, 8), (1, 0), (1, 3), (8, 1)])
def test_gather_of_strided_rows(lib, dtype, shift, pad):
    rng = np.random.default_rng(3)
    p, want = make_plan(lib, rng, 40, 2, 6, "dropped")
    store = torch.randn(40 * (512 + pad) + shift, device=dev).to(dtype)
    x = store[shift:].view(40, 512 + pad)[:, :512]
    got = lib.expert_gather(x, p)
    assert torch.equal(got, lib.expert_gather(x.contiguous(), p))
    row = want[3]
    ref = np.where((row >= 0)[:, None], np64(x)[np.maximum(row, 0) // 2], 0)
    assert np.array_equal(np64(got), ref)


# ------------------------------------------------------------------ gather to MX
def bf16_values(rng, tokens, cols, special=True):
    x = rng.standard_normal((tokens, cols)) * np.exp2(rng.integers(-12, 12, size=(tokens, 1)))
    x = torch.from_numpy(x).to(BF)
    if special:
        flat = x.view(-1)
        n = flat.numel()
        for v in (float("nan"), float("inf"), -float("inf"), -0.0, 0.0, 1e-40, 3e38):
            flat[torch.from_numpy(rng.integers(0, n, size=max(1, n // 2000)))] = v
    return x.to(dev)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2", "e2m1"])
@pytest.mark.parametrize("orientation", ["row", "col", "dual"])
@pytest.mark.parametrize("scale,layout", [("floor", "canonical"), ("ceil", "mma")])
@pytest.mark.parametrize("tokens,top,experts,cols,align", [(1, 1, 1, 128, 128), (1, 8, 64, 256, 128), (300, 2, 5, 384, 256),
                                                           (1000, 3, 16, 640, 128)])
def test_gather_to_mx(lib, tokens, top, experts, cols, align, scale, layout, orientation, fmt):
    """Byte for byte the quantizer's output (which the oracle pins) for the gathered rows."""
    rng = np.random.default_rng(cols + tokens)
    p, _ = make_plan(lib, rng, tokens, top, experts, "dropped" if tokens > 1 else "even", align)
    x = bf16_values(rng, tokens, cols)
    got = lib.mx_expert_gather(x, p, fmt, orientation, scale, layout)
    want = lib.mx_quantize(lib.expert_gather(x, p), fmt, orientation, scale, sf_layout=layout)
    for g, w, name in zip(got, want, ("q_row", "s_row", "q_col", "s_col")):
        assert (g is None) == (w is None) and (g is None or torch.equal(g, w)), name


@pytest.mark.parametrize("cols", [32, 96, 160, 224])
def test_gather_to_mx_of_narrow_and_strided_rows(lib, cols):
    """Columns that end inside a tile, in rows that are wider than what is read."""
    rng = np.random.default_rng(cols)
    p, _ = make_plan(lib, rng, 77, 2, 5, "dropped")
    wide = bf16_values(rng, 77, cols + 40)
    x = wide[:, 8:8 + cols]
    got = lib.mx_expert_gather(x, p, "e4m3", "dual", "floor", "canonical")
    want = lib.mx_quantize(lib.expert_gather(x, p), "e4m3", "dual", "floor")
    assert all(torch.equal(g, w) for g, w in zip(got, want))


# ------------------------------------------------------------------ combine
def inputs(rng, p, cols, dtype, wtype, fill=0.0):
    """Rows whose padding holds `fill`, and gate weights whose dropped slots hold NaN."""
    rows = torch.randn(p.rows, cols, generator=torch.Generator().manual_seed(cols)).to(dtype).to(dev)
    rows[p.row_slot < 0] = fill
    w = torch.rand(p.tokens, p.top, generator=torch.Generator().manual_seed(1)).to(wtype).to(dev)
    w[p.slot_row < 0] = float("nan")
    return rows, w


def combine64(rows, w, slot_row):
    """(sum, sum of magnitudes) in float64."""
    r = np64(rows)
    live = slot_row >= 0
    wv = np.where(live, 1.0 if w is None else np64(w), 0.0)
    at = np.maximum(slot_row, 0)
    y = np.zeros((slot_row.shape[0], r.shape[1]))
    m = np.zeros_like(y)
    for j in range(slot_row.shape[1]):
        term = np.where(live[:, j, None], r[at[:, j]], 0.0) * wv[:, j, None]
        y += term
        m += np.abs(term)
    return y, m


SHAPES = [(1, 1, 1, 1), (1, 8, 64, 4096), (5, 2, 3, 7), (33, 3, 5, 1021), (130, 2, 4, 1024), (70, 4, 8, 5000), (64, 33, 40, 264)]


@pytest.mark.parametrize("pattern", ["even", "dropped", "none", "one"])
@pytest.mark.parametrize("dtype,out,wtype", [(BF, BF, F32), (BF, F32, BF), (F32, BF, F32), (F32, F32, F32), (BF, BF, None)])
@pytest.mark.parametrize("tokens,top,experts,cols", SHAPES)
def test_combine(lib, tokens, top, experts, cols, dtype, out, wtype, pattern):
    rng = np.random.default_rng(cols)
    p, want = make_plan(lib, rng, tokens, top, experts, pattern)
    rows, w = inputs(rng, p, cols, dtype, wtype or F32, float("nan"))
    w = None if wtype is None else w
    y = lib.expert_combine(rows, p, w, out)
    ref, mag = combine64(rows.nan_to_num(0.0), None if w is None else w.nan_to_num(0.0), want[2])
    # top fused steps in float32, each off by half a step of a partial sum (at most mag), then one rounding
    tol = top * 2.0 ** -24 * mag * (1 + 1e-5)
    tol = tol + half_ulp(out, ref, tol)
    assert y.dtype == out and np.all(np.abs(np64(y) - ref) <= tol)
    assert np.all(np64(y)[(want[2] < 0).all(1)] == 0)


@pytest.mark.parametrize("pattern", ["even", "dropped"])
@pytest.mark.parametrize("dtype,out,wtype", [(BF, BF, F32), (BF, F32, BF), (F32, BF, BF), (F32, F32, None)])
@pytest.mark.parametrize("tokens,top,experts,cols", [(2100, 2, 7, 1024), (2200, 3, 5, 1021), (4099, 1, 3, 515), (70000, 2, 64, 32),
                                                     (30011, 5, 9, 77), (513, 2, 4, 4104), (9001, 2, 4, 264)])
def test_combine_of_many_tokens(lib, tokens, top, experts, cols, dtype, out, wtype, pattern):
    """Sizes of the ring of asynchronous copies, every lane group and alignment of it."""
    rng = np.random.default_rng(cols)
    p, want = make_plan(lib, rng, tokens, top, experts, pattern)
    rows, w = inputs(rng, p, cols, dtype, wtype or F32, float("nan"))
    if wtype == BF:                                  # weights that start inside a 4-byte word
        store = torch.empty(w.numel() + 1, dtype=BF, device=dev)
        store[1:] = w.view(-1)
        w = store[1:].view(w.shape)
    w = None if wtype is None else w
    y = lib.expert_combine(rows, p, w, out)
    ref, mag = combine64(rows.nan_to_num(0.0), None if w is None else w.nan_to_num(0.0), want[2])
    tol = top * 2.0 ** -24 * mag * (1 + 1e-5)
    tol = tol + half_ulp(out, ref, tol)
    assert np.all(np.abs(np64(y) - ref) <= tol)
    if cols % 8 and dtype == BF:                     # rows that start elsewhere in their words
        store = torch.empty(p.rows * (cols + 3) + 5, dtype=BF, device=dev)
        shifted = store[5:].view(p.rows, cols + 3)[:, :cols]
        shifted.copy_(rows)
        assert torch.equal(lib.expert_combine(shifted, p, w, out), y)


def test_combine_of_strided_and_shifted_rows(lib):
    rng = np.random.default_rng(5)
    p, _ = make_plan(lib, rng, 50, 2, 4, "dropped")
    for dtype in (BF, F32):
        for shift, pad, cols in ((0, 16, 512), (1, 0, 512), (2, 6, 512), (1, 1, 511)):
            store = torch.randn(p.rows * (cols + pad) + shift, device=dev).to(dtype)
            rows = store[shift:].view(p.rows, cols + pad)[:, :cols]
            w = torch.rand(50, 2, device=dev)
            assert torch.equal(lib.expert_combine(rows, p, w), lib.expert_combine(rows.contiguous(), p, w))
            dstore = torch.randn(50 * (cols + pad) + shift, device=dev).to(dtype)
            dy = dstore[shift:].view(50, cols + pad)[:, :cols]
            got = lib.expert_combine_backward(dy, rows, p, w)
            want = lib.expert_combine_backward(dy.contiguous(), rows.contiguous(), p, w)
            assert torch.equal(got[0], want[0])
            ref = (np64(dy)[:, None] * np64(rows)[np.maximum(p.slot_row.cpu().numpy(), 0)])
            live = p.slot_row.cpu().numpy() >= 0
            tol = cols * 2.0 ** -24 * np.abs(ref).sum(2)
            assert np.all(np.abs(np64(got[1]) - np.where(live, ref.sum(2), 0)) <= tol)


# ------------------------------------------------------------------ combine, backward
@pytest.mark.parametrize("pattern", ["even", "dropped", "none", "one"])
@pytest.mark.parametrize("dtype,dytype,wtype", [(BF, BF, F32), (BF, F32, BF), (F32, BF, F32), (F32, F32, F32)])
@pytest.mark.parametrize("tokens,top,experts,cols", SHAPES)
def test_combine_backward(lib, tokens, top, experts, cols, dtype, dytype, wtype, pattern):
    rng = np.random.default_rng(cols)
    p, want = make_plan(lib, rng, tokens, top, experts, pattern)
    rows, w = inputs(rng, p, cols, dtype, wtype, float("nan"))
    dy = torch.randn(tokens, cols, generator=torch.Generator().manual_seed(2)).to(dytype).to(dev)
    drows, dw = lib.expert_combine_backward(dy, rows, p, w)
    assert drows.dtype == dtype and dw.dtype == F32
    live, at = want[2] >= 0, np.maximum(want[2], 0)
    ref = np.zeros((p.rows, cols))
    wv = np.where(live, np64(w), 0.0)
    for j in range(top):
        ref[at[live[:, j], j]] = (np64(dy) * wv[:, j, None])[live[:, j]]
    tol = 2.0 ** -24 * np.abs(ref)
    assert np.all(np.abs(np64(drows) - ref) <= tol + half_ulp(dtype, ref, tol) * (ref != 0))
    prod = np64(dy)[:, None] * np.where(live[:, :, None], np64(rows)[at], 0.0)
    # a term passes cols / 256 sums of its thread at most (and 8 within a vector), 5 of its warp, 8 of the CTA; one product
    steps = cols // 256 + 1 + 8 + 5 + 8 + 1
    assert np.all(np.abs(np64(dw) - prod.sum(2)) <= steps * 2.0 ** -24 * np.abs(prod).sum(2))
    assert np.all(np64(dw)[~live] == 0)
    again = lib.expert_combine_backward(dy, rows, p, w)
    assert torch.equal(again[0], drows) and torch.equal(again[1], dw)


@pytest.mark.parametrize("pattern", ["even", "dropped"])
@pytest.mark.parametrize("dtype,wtype", [(BF, F32), (BF, BF), (F32, BF), (F32, F32)])
@pytest.mark.parametrize("tokens,top,experts,cols", [(4100, 2, 7, 1024), (4700, 1, 5, 904), (2100, 9, 30, 2048), (1100, 3, 4, 4096),
                                                     (1030, 2, 4, 4104), (520, 17, 20, 8192), (520, 2, 3, 8200), (8200, 8, 11, 520)])
def test_combine_backward_of_many_tokens(lib, tokens, top, experts, cols, dtype, wtype, pattern):
    """Sizes of the ring of asynchronous copies, and the first ones beyond it."""
    rng = np.random.default_rng(cols)
    p, want = make_plan(lib, rng, tokens, top, experts, pattern)
    rows, w = inputs(rng, p, cols, dtype, wtype, float("nan"))
    if wtype == BF:                                  # weights that start inside a 4-byte word
        store = torch.empty(w.numel() + 1, dtype=BF, device=dev)
        store[1:] = w.view(-1)
        w = store[1:].view(w.shape)
    dy = torch.randn(tokens, cols, generator=torch.Generator().manual_seed(2)).to(dtype).to(dev)
    drows, dw = lib.expert_combine_backward(dy, rows, p, w)
    # float64 on the GPU, slot by slot
    slot = torch.from_numpy(want[2]).to(dev)
    ref = torch.zeros(p.rows, cols, dtype=torch.float64, device=dev)
    steps = cols // 256 + 1 + 8 + 5 + 8 + 1
    for j in range(top):
        live = slot[:, j] >= 0
        at, d = slot[live, j], dy[live].double()
        ref[at] = d * w[live, j].double()[:, None]
        prod = d * rows[at].double()
        assert bool(((dw[live, j].double() - prod.sum(1)).abs() <= steps * 2.0 ** -24 * prod.abs().sum(1)).all())
        assert not bool(dw[~live, j].any())
    half = 2.0 ** -9 if dtype == BF else 2.0 ** -24
    # one rounding of the product to float32 and one to the rows' type, each at most half a step of the value's binade
    assert bool(((drows.double() - ref).abs() <= ref.abs() * (2 * half + 2.0 ** -23) + 2.0 ** -130).all())
    again = lib.expert_combine_backward(dy, rows, p, w)
    assert torch.equal(again[0], drows) and torch.equal(again[1], dw)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("cols", [11, 128, 1021, 4096])
@pytest.mark.parametrize("tokens", [37, 1300, 5000])
def test_gather_bit_for_bit(lib, tokens, cols, dtype):
    """Fewer and more tokens than fill the GPU, every bit pattern (NaN, too), rows
    with gaps between them."""
    g = torch.Generator(device=dev).manual_seed(tokens + cols)
    bits, size = (torch.int16, 2) if dtype == BF else (torch.int32, 4)
    x = torch.randint(-2 ** 15, 2 ** 15, (tokens, (cols + 5) * size // 2), generator=g, device=dev).to(torch.int16).view(dtype)[:, :cols]
    plan = lib.expert_sort(torch.randint(-1, 7, (tokens, 3), generator=g, device=dev), 7, 128)
    got = lib.expert_gather(x, plan).view(bits)
    want = torch.zeros(plan.rows, cols, dtype=bits, device=dev)
    live = plan.row_slot >= 0
    want[live] = x.contiguous().view(bits)[(plan.row_slot[live] // 3).long()]
    assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("gap", [0, 8])
@pytest.mark.parametrize("tokens,cols", [(40, 1024), (1000, 128), (30000, 128), (5000, 1024), (4001, 2080), (5000, 4096)])
def test_gather_of_aligned_rows_bit_for_bit(lib, tokens, cols, gap, dtype):
    """Rows of whole words, on both sides of where slots go apart: a token read
    once and stored to the rows of all its slots, in one stretch and in several."""
    g = torch.Generator(device=dev).manual_seed(tokens + cols)
    bits, size = (torch.int16, 2) if dtype == BF else (torch.int32, 4)
    x = torch.randint(-2 ** 15, 2 ** 15, (tokens, (cols + gap) * size // 2), generator=g, device=dev).to(torch.int16).view(dtype)[:, :cols]
    assert x.data_ptr() % 16 == 0 and x.stride(0) * size % 16 == 0 and cols * size % 16 == 0
    plan = lib.expert_sort(torch.randint(-1, 7, (tokens, 3), generator=g, device=dev), 7, 128)
    got = lib.expert_gather(x, plan).view(bits)
    want = torch.zeros(plan.rows, cols, dtype=bits, device=dev)
    live = plan.row_slot >= 0
    want[live] = x.contiguous().view(bits)[(plan.row_slot[live] // 3).long()]
    assert torch.equal(got, want)


@pytest.mark.parametrize("cols", [512, 4096, 509, 2049])
@pytest.mark.parametrize("dtype,dytype", [(BF, F32), (F32, BF)])
def test_combine_backward_of_few_tokens(lib, cols, dtype, dytype):
    """A few tokens and, among thousands of them, the same ones: what each gets is
    the same, but for the order of a sum where rows lie differently."""
    many, few, top, E = 4200, 37, 5, 6
    g = torch.Generator(device=dev).manual_seed(cols)
    experts = torch.randint(-1, E, (many, top), generator=g, device=dev)
    rows_of = torch.randn(many * top, cols, generator=g, device=dev).to(dtype)       # by slot
    dy = torch.randn(many, cols + 3, generator=g, device=dev).to(dytype)[:, :cols]
    w = torch.rand(many, top, generator=g, device=dev)
    got = []
    for T in (few, many):
        plan = lib.expert_sort(experts[:T].contiguous(), E, 128)
        live = plan.slot_row >= 0
        at = plan.slot_row[live].long()
        rows = torch.zeros(plan.rows, cols, dtype=dtype, device=dev)
        rows[at] = rows_of[: T * top].view(T, top, cols)[live]
        drows, dw = lib.expert_combine_backward(dy[:T], rows, plan, w[:T].contiguous())
        pad = torch.ones(plan.rows, dtype=torch.bool, device=dev)
        pad[at] = False
        assert not drows[pad].any() and not dw[~live].any()
        mine = live.clone()
        mine[few:] = False
        got.append((drows[plan.slot_row[mine].long()], dw[:few]))
    (da, wa), (db, wb) = got
    assert torch.equal(da, db)
    # a sum of n products in any order: n half steps of the sum of magnitudes, twice
    mag = (dy[:few, None, :].double() * rows_of[: few * top].view(few, top, cols).double()).abs().sum(2)
    assert ((wa - wb).abs().double() <= 2 * cols * 2.0 ** -24 * mag).all()


@pytest.mark.parametrize("gap", [0, 8])
@pytest.mark.parametrize("dtype,dytype", [(BF, BF), (F32, F32), (BF, F32), (F32, BF)])
@pytest.mark.parametrize("tokens,top,cols", [(2000, 2, 128), (2000, 5, 256), (1000, 3, 512), (2000, 2, 1024), (2000, 5, 1024),
                                             (700, 8, 2048), (500, 3, 4096), (300, 2, 8192), (4000, 5, 512), (6000, 4, 520)])
def test_combine_backward_of_aligned_rows(lib, tokens, top, cols, dtype, dytype, gap):
    """Aligned rows, several slots to a token and tokens enough that a team takes
    all of a token's slots: dy in registers over pairs of slots, an odd one among
    them, rows longer than that, and dy of another type than the rows."""
    g = torch.Generator(device=dev).manual_seed(tokens + cols)
    plan = lib.expert_sort(torch.randint(-1, 6, (tokens, top), generator=g, device=dev), 6, 128)
    rows = torch.randn(plan.rows, cols + gap, generator=g, device=dev).to(dtype)[:, :cols]
    rows[plan.row_slot < 0] = float("nan")                            # padding is not looked at
    dy = torch.randn(tokens, cols + gap, generator=g, device=dev).to(dytype)[:, :cols]
    w = torch.rand(tokens, top, generator=g, device=dev)
    drows, dw = lib.expert_combine_backward(dy, rows, plan, w)
    ref = torch.zeros(plan.rows, cols, dtype=torch.float64, device=dev)
    # a product, sums of 8 within a vector, of a thread's vectors, of 32 lanes, of 8 warps
    steps = 1 + 3 + cols // 256 + 1 + 5 + 8
    for j in range(top):
        live = plan.slot_row[:, j] >= 0
        at, d = plan.slot_row[live, j].long(), dy[live].double()
        ref[at] = d * w[live, j].double()[:, None]
        prod = d * rows[at].double()
        assert bool(((dw[live, j].double() - prod.sum(1)).abs() <= steps * 2.0 ** -24 * 1.001 * prod.abs().sum(1)).all())
        assert not bool(dw[~live, j].any())
    # the product rounded to float32, and once more to bf16
    tol = ref.abs() * (2.0 ** -24 + (2.0 ** -8 * (1 + 2.0 ** -24) if dtype == BF else 0.0))
    assert bool(((drows.double() - ref).abs() <= tol).all())
    again = lib.expert_combine_backward(dy, rows, plan, w)
    assert torch.equal(again[0], drows) and torch.equal(again[1], dw)


def test_gradients_against_differences(lib):
    """The sum is linear in the rows and in the weights: a difference over a
    step h is the gradient up to the float32 rounding of both sums, 4 steps of
    half an ulp each of a token's magnitude."""
    rng = np.random.default_rng(11)
    p, want = make_plan(lib, rng, 20, 3, 4, "dropped")
    rows, w = inputs(rng, p, 64, F32, F32)
    w = w.nan_to_num(0.5)
    g = torch.randn(20, 64, device=dev)
    drows, dw = lib.expert_combine_backward(g, rows, p, w)
    loss = lambda r, ww: (np64(lib.expert_combine(r, p, ww)) * np64(g)).sum()
    _, mag = combine64(rows, w, want[2])
    noise = 2 * 4 * 2.0 ** -24 * np.abs(np64(g) * (mag + 1)).sum()
    for _ in range(10):
        t, j = rng.integers(20), rng.integers(3)
        h = torch.zeros_like(w)
        h[t, j] = 0.25
        assert abs((loss(rows, w + h) - loss(rows, w - h)) / 0.5 - float(dw[t, j])) <= 2 * noise
        r, c = rng.integers(p.rows), rng.integers(64)
        h = torch.zeros_like(rows)
        h[r, c] = 0.25
        assert abs((loss(rows + h, w) - loss(rows - h, w)) / 0.5 - float(drows[r, c])) <= 2 * noise
    # the gather's gradient is the combine without weights
    x = torch.randn(20, 64, device=dev)
    G = torch.randn(p.rows, 64, device=dev)
    dx = lib.expert_combine(G, p)
    for _ in range(10):
        t, c = rng.integers(20), rng.integers(64)
        up, down = x.clone(), x.clone()
        up[t, c], down[t, c] = 1.0, -1.0
        d = (np64(lib.expert_gather(up, p) - lib.expert_gather(down, p)) * np64(G)).sum() / 2
        assert abs(d - float(dx[t, c])) <= 3 * 2.0 ** -24 * 3 * np.abs(np64(G)).max()


def test_offsets_that_pass_32_bits(lib):
    """Tensors of more than 2^31 elements: the last rows and columns are where they belong."""
    tokens, cols = 300000, 8192
    e = torch.arange(tokens, device=dev, dtype=torch.int32).view(-1, 1) % 3
    p = lib.expert_sort(e, 3)
    x = torch.empty(tokens, cols, dtype=BF, device=dev)
    x.copy_((torch.arange(tokens, device=dev) % 251)[:, None])
    x[:, -1] = 2.0
    rows = lib.expert_gather(x, p)
    at = p.slot_row.view(-1).long()
    assert torch.equal(rows[at[-5000:]], x[-5000:]) and torch.equal(rows[at[:100]], x[:100]) and not rows[-1].any()
    q, s, qT, sT = lib.mx_expert_gather(x, p, "e4m3", "dual", sf_layout="mma")
    lo = int(p.offsets[2]) + 128 * 700               # a stretch of the last expert
    part = lib.mx_quantize(rows[lo:lo + 256].contiguous(), "e4m3", "dual", sf_layout="canonical")
    assert torch.equal(q[lo:lo + 256], part[0]) and torch.equal(qT[:, lo:lo + 256], part[2])
    assert p.rows * cols > 2 ** 31
    del q, s, qT, sT, part
    w = torch.full((tokens, 1), 0.5, device=dev)
    y = lib.expert_combine(rows, p, w)
    assert torch.equal(y[-5000:], x[-5000:] * 0.5)
    del y
    d, dw = lib.expert_combine_backward(x, rows, p, w)
    assert torch.equal(d[at[-5000:]], x[-5000:] * 0.5) and not d[-1].any()
    # a row's products are whole numbers: (cols - 1) v^2 + 4 up to 2^29, off by half a step of each partial sum
    v = (torch.arange(tokens, device=dev) % 251).double()
    want = (cols - 1) * v * v + 4
    assert bool(((dw.view(-1).double() - want).abs() <= 64 * 2.0 ** -24 * want).all())
    del d, rows
    drop = lib.dropout(x, 0.5, 7, residual=x)
    tail = lib.dropout(x[-1000:].contiguous(), 0.5, 7, (tokens - 1000) * cols // 4, residual=x[-1000:].contiguous())
    assert torch.equal(drop[-1000:], tail)


def test_a_wrong_plan_reads_and_writes_within_bounds(lib):
    """Indices beyond the rows or tokens are passed over (a plan changed by hand)."""
    rng = np.random.default_rng(6)
    p, _ = make_plan(lib, rng, 16, 2, 4)
    p.slot_row.fill_(2 ** 31 - 1)
    p.row_slot.fill_(2 ** 31 - 1)
    for off, n in ((2 ** 31 - 1, 2 ** 31 - 1), (-(2 ** 31), -(2 ** 31)), (2 ** 31 - 1, -(2 ** 31)), (64, -65)):
        p.offsets.fill_(off)
        p.counts.fill_(n)
        lib.expert_gather(torch.zeros(16, 129, device=dev), p)
    rows = torch.randn(p.rows, 128, device=dev).to(BF)
    assert not lib.expert_combine(rows, p).any()
    _, dw = lib.expert_combine_backward(rows[:16], rows, p, torch.ones(16, 2, device=dev))
    assert not dw.any()
    lib.expert_gather(rows[:16], p)
    q = lib.mx_expert_gather(rows[:16], p, "e4m3", "dual")
    assert not q[0].any() and not q[2].any()
    # the rings, and a plan of no rows at all
    p, _ = make_plan(lib, rng, 4200, 1, 4)
    rows = torch.randn(p.rows, 1024, device=dev).to(BF)
    for r in (2 ** 31 - 1, -(2 ** 31), p.rows):
        p.slot_row.fill_(r)
        assert not lib.expert_combine(rows, p, torch.ones(4200, 1, device=dev)).any()
        assert not lib.expert_combine(rows[:, 1:], p, torch.ones(4200, 1, device=dev)).any()
        d, dw = lib.expert_combine_backward(rows[:4200], rows, p, torch.ones(4200, 1, device=dev))
        assert not dw.any()
    p.slot_row.zero_()
    dw, w, zero = torch.ones(4200, 1, device=dev), torch.ones(4200, 1, device=dev), torch.zeros(8, dtype=torch.int32, device=dev)
    y = torch.ones(4200, 1024, dtype=BF, device=dev)
    stream = torch.cuda.current_stream().cuda_stream
    at = p.slot_row.data_ptr()
    assert lib.load().mxq_expert_combine_backward(rows.data_ptr(), 1024, 0, None, 1024, 0, 0, 1024, at, 4200, 1, zero.data_ptr(),
                                                  zero.data_ptr(), 4, w.data_ptr(), 1, None, dw.data_ptr(), stream) == 0
    assert lib.load().mxq_expert_combine(None, 0, 1024, 1024, 0, at, 4200, 1, w.data_ptr(), 1, y.data_ptr(), 0, stream) == 0
    assert not dw.any() and not y.any()
