"""GPU tests of layer_norm, mx_layer_norm and layer_norm_backward against the
formulas in float64, on the bits that the kernels read.

Tolerances, with u = 2^-24 the float32 rounding unit: a sum over a row is a
tree of at most 20 additions for rows held in registers (five in a thread's
vectors, five over the vectors, two times five over lanes and warps), and
cols / 1024 more for the rows that a CTA loops over; a column sum adds a
thread's rows, then at most 16 groups and 608 / 8 parts.  Every bound below
counts roundings that way and multiplies them by the magnitudes that they act
on; the rounding to the result's type adds half an ulp."""

import numpy as np
import pytest
import torch

from oracle import formats as F
from oracle import mx as omx
from tests.rounding import half_ulp

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
dev = torch.device("cuda")
BF, F32 = torch.bfloat16, torch.float32
FMT = {"e4m3": F.E4M3, "e5m2": F.E5M2, "e2m1": F.E2M1}


def make(shape, dtype, seed, scale=1.0, offset=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale + offset).to(dtype)


def d(t):
    return t.detach().cpu().double().numpy()


def forward_ref(x, w, b, eps=1e-5):
    """y, mean, rstd and the absolute error bound of each, float64."""
    x = d(x)
    n = x.shape[1]
    w = np.ones(n) if w is None else d(w)
    b = np.zeros(n) if b is None else d(b)
    mean = x.mean(1, keepdims=True)
    dev_ = x - mean
    var = (dev_ ** 2).mean(1, keepdims=True)
    rstd = 1.0 / np.sqrt(var + eps)
    y = dev_ * rstd * w + b
    k = 24 + n / 1024
    e_mean = k * U * np.abs(x).mean(1, keepdims=True)
    # rstd moves by half the relative error of var + eps: the sum's roundings, the deviations' and the mean's square
    e_rel = (k + 4) * U + e_mean ** 2 / (var + eps)
    e_y = np.abs(w) * rstd * (e_mean + U * np.abs(dev_)) + np.abs(w * dev_ * rstd) * (e_rel + 4 * U) + 2 * U * (np.abs(y) + np.abs(b))
    return y, mean[:, 0], rstd[:, 0], e_y, e_mean[:, 0], (e_rel * rstd)[:, 0]


def check_forward(lib, x, w, b, out_dtype=None, eps=1e-5):
    y, mean, rstd = lib.layer_norm(x, w, b, eps, out_dtype=out_dtype)
    ry, rm, rr, ey, em, er = forward_ref(x, w, b, eps)
    assert y.dtype == (out_dtype or x.dtype) and y.shape == x.shape and y.is_contiguous()
    assert (np.abs(d(mean) - rm) <= em + U * np.abs(rm)).all()
    assert (np.abs(d(rstd) - rr) <= er).all()
    assert (np.abs(d(y) - ry) <= ey + half_ulp(y.dtype, ry, ey)).all()


SHAPES = [(1, 1), (3, 1), (1, 4096), (5, 7), (1, 8), (2, 31), (9, 32), (17, 33), (4, 255), (3, 256), (8, 1000), (7, 1021),
          (5, 1024), (3, 1032), (2, 2049), (3, 4104), (2, 8191), (2, 8192), (2, 14336), (2, 16385), (1, 32768),
          (2, 32767), (2, 32769), (1, 40000)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("xt,yt", [(BF, BF), (F32, F32), (F32, BF), (BF, F32)])
def test_forward_shapes_and_types(lib, rows, cols, xt, yt):
    x = make((rows, cols), xt, rows * 7 + cols, 2.0, 0.5).to(dev)
    w = make((cols,), BF if cols % 2 else F32, 1, 0.3, 1.0).to(dev)
    b = make((cols,), F32 if cols % 3 else BF, 2, 0.3).to(dev)
    check_forward(lib, x, w, b, yt)


@pytest.mark.parametrize("rows,cols", [(5, 520), (300, 64), (3, 4096)])
def test_forward_without_weight_or_bias(lib, rows, cols):
    x = make((rows, cols), BF, 3).to(dev)
    w = make((cols,), BF, 4, 0.1, 1.0).to(dev)
    check_forward(lib, x, None, None)
    check_forward(lib, x, w, None)
    check_forward(lib, x, None, w)


@pytest.mark.parametrize("cols", [256, 1024, 2050])
@pytest.mark.parametrize("shift", [0, 1, 3, 8])
def test_forward_strided_rows_and_odd_bases(lib, cols, shift):
    """A slice of a wider tensor: row stride beyond cols, bases off 16 bytes."""
    for dt in (BF, F32):
        wide = make((6, cols + 13), dt, 5).to(dev)
        x = wide[1:5, shift:shift + cols]
        wb = make((2, cols + 1), dt, 6, 0.1, 1.0).to(dev)
        check_forward(lib, x, wb[0, 1:], wb[1, :cols])


def test_forward_large_mean_does_not_cancel(lib):
    """Spread 1 around 1000: one-pass sums of squares would lose the variance."""
    x = make((4, 4096), F32, 7, 1.0, 1000.0).to(dev)
    check_forward(lib, x, None, None)
    assert torch.allclose(lib.layer_norm(x)[2].cpu(), torch.ones(4), rtol=0.05)


def test_forward_constant_zero_and_empty_rows(lib):
    x = torch.zeros(3, 640, device=dev)
    x[1] = 7.25
    y, mean, rstd = lib.layer_norm(x)
    assert (y == 0).all() and mean.tolist() == [0.0, 7.25, 0.0]
    assert torch.allclose(rstd.cpu(), torch.full((3,), 1e-5).rsqrt())
    y, mean, rstd = lib.layer_norm(torch.empty(0, 640, device=dev, dtype=BF))
    assert y.shape == (0, 640) and mean.numel() == 0 and rstd.numel() == 0


@pytest.mark.parametrize("rows", [3, 6000])
def test_forward_variance_at_the_ends_of_float32(lib, rows):
    """eps 0 on constant rows: rstd is infinite, y NaN (0 * inf), as the formula
    says.  Variances beyond float32: rstd 0 and y = bias."""
    x = torch.full((rows, 1024), 2.0, device=dev)
    y, mean, rstd = lib.layer_norm(x, eps=0.0)
    assert (mean == 2).all() and rstd.isinf().all() and y.isnan().all()
    x[:, ::2] = 1e25
    b = torch.full((1024,), 0.5, device=dev)
    y, mean, rstd = lib.layer_norm(x, None, b)
    assert (rstd == 0).all() and (y == 0.5).all()


@pytest.mark.parametrize("cols", [640, 4096, 2049, 33000])
def test_forward_nonfinite_rows_stay_alone(lib, cols):
    """NaN and infinities make their own row NaN and touch no other."""
    x = make((5, cols), F32, 8).to(dev)
    clean = lib.layer_norm(x)[0]
    x[1, 3] = float("nan")
    x[3, cols - 1] = float("inf")
    y = lib.layer_norm(x)[0]
    assert y[1].isnan().all() and y[3].isnan().all()
    for r in (0, 2, 4):
        assert torch.equal(y[r], clean[r])


def test_forward_runs_on_the_current_stream(lib):
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        x = make((64, 4096), F32, 9).to(dev)
        torch.cuda._sleep(20_000_000)
        x.mul_(3.0)
        y, mean, rstd = lib.layer_norm(x)
        q = lib.mx_layer_norm(x.bfloat16(), orientation="dual")
    s.synchronize()
    ry, *_ , = forward_ref(x, None, None)
    assert np.abs(d(y) - ry).max() < 1e-4
    assert q[0].any() and q[2].any()


# ------------------------------------------------------------------ straight to MX
def check_blocks(q, s, y, ey, fmt, mode, what):
    """Codes q and canonical scales s of the row blocks of y known to +-ey:
    each scale is that of an amax in the known range, and each code lies
    between the codes of the range's ends under that scale (rounding is
    monotone)."""
    f = FMT[fmt]
    R, C = y.shape
    if f.nbits == 4:
        q = F.unpack_fp4(q)
    lo_a = np.maximum(np.abs(y) - ey, 0).reshape(R, C // 32, 32).max(2)
    hi_a = (np.abs(y) + ey).reshape(R, C // 32, 32).max(2)
    e = s.astype(np.int64) - 127
    assert (e >= omx.scale_exponent(lo_a, f, mode)).all() and (e <= omx.scale_exponent(hi_a, f, mode)).all(), what
    x2 = np.repeat(2.0 ** -e.astype(np.float64), 32, axis=1)
    got = F.decode(f, q)
    assert (got >= F.decode(f, F.encode_rne_sat(f, (y - ey) * x2))).all(), what
    assert (got <= F.decode(f, F.encode_rne_sat(f, (y + ey) * x2))).all(), what
    # and they are the quantization of y itself wherever no boundary lies in the range: nearly everywhere
    same = F.decode(f, F.encode_rne_sat(f, y * x2)) == got
    assert same.mean() > 0.999, what


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2", "e2m1"])
@pytest.mark.parametrize("orient", ["row", "col", "dual"])
@pytest.mark.parametrize("rows,cols,xt,sf", [(32, 32, BF, "canonical"), (96, 416, F32, "canonical"), (128, 128, BF, "mma"),
                                             (64, 1056, BF, "canonical"), (256, 640, F32, "mma"), (128, 2048, F32, "mma"),
                                             (128, 4224, BF, "mma"), (32, 8192, BF, "canonical"),
                                             (32, 8224, BF, "canonical"), (64, 4128, F32, "canonical"),
                                             (32, 14336, BF, "canonical")])
def test_mx_against_the_range_of_y(lib, fmt, orient, rows, cols, xt, sf):
    mode = "ceil" if (rows + cols) % 64 else "floor"
    x = make((rows, cols), xt, rows + cols, 2.0, 0.3).to(dev)
    x[:, 5] *= 30
    w = make((cols,), F32 if xt == BF else BF, 1, 0.3, 1.0).to(dev)
    b = make((cols,), BF, 2, 0.3).to(dev)
    q, s, qT, sT, mean, rstd = lib.mx_layer_norm(x, w, b, 1e-5, fmt, orient, mode, sf)
    ry, rm, rr, ey, em, er = forward_ref(x, w, b)
    assert (np.abs(d(mean) - rm) <= em + U * np.abs(rm)).all() and (np.abs(d(rstd) - rr) <= er).all()
    m = {"floor": omx.FLOOR, "ceil": omx.CEIL}[mode]
    sides = {"row": (q, s, ry, ey), "col": (qT, sT, ry.T, ey.T)}
    for side, (qq, ss, y, e) in sides.items():
        if orient not in (side, "dual"):
            assert qq is None and ss is None
            continue
        ss = ss.cpu().numpy()
        if sf == "mma":
            ss = omx.sf_from_mma(ss, y.shape[0], y.shape[1] // 32)
        check_blocks(qq.cpu().numpy(), ss, y, e, fmt, m, side)


def test_mx_long_rows(lib):
    """Beyond one CTA's registers (32768) rows quantize after a pass for their statistics."""
    x = make((32, 32800), BF, 3).to(dev)
    for orient in ("row", "dual"):
        q, s, qT, sT, mean, rstd = lib.mx_layer_norm(x, orientation=orient)
        ry, _, _, ey, _, _ = forward_ref(x, None, None)
        check_blocks(q.cpu().numpy(), s.cpu().numpy(), ry, ey, "e4m3", omx.FLOOR, "row")
        if orient == "dual":
            check_blocks(qT.cpu().numpy(), sT.cpu().numpy(), ry.T, ey.T, "e4m3", omx.FLOOR, "col")


def test_mx_exact_values(lib):
    """Rows of +-1 have mean 0 and variance 1: with eps 0 y = +-w + b exactly, so every byte is the oracle's."""
    cols = 2048
    x = torch.ones(64, cols)
    x[:, ::2] = -1
    x = x[:, torch.randperm(cols, generator=torch.Generator().manual_seed(0))]
    w = make((cols,), BF, 1, 1.0).to(dev)
    b = make((cols,), BF, 2, 1.0)
    b = (b.float() * 0).to(BF).to(dev)
    for fmt in FMT:
        for mode in ("floor", "ceil"):
            q, s, qT, sT, _, rstd = lib.mx_layer_norm(x.to(dev).to(BF), w, b, 0.0, fmt, "dual", mode)
            assert (rstd == 1).all()
            ref = omx.quantize(d(x) * d(w), FMT[fmt], omx.DUAL, {"floor": omx.FLOOR, "ceil": omx.CEIL}[mode])
            # the fused multiply-add gives w*h + 0: a negative zero becomes +0, so compare values
            for got, want in ((q, ref["q_row"]), (qT, ref["q_col"])):
                g, r = got.cpu().numpy(), want
                if fmt == "e2m1":
                    g, r = F.unpack_fp4(g), F.unpack_fp4(r)
                assert np.array_equal(F.decode(FMT[fmt], g), F.decode(FMT[fmt], r))
            assert np.array_equal(s.cpu().numpy(), ref["s_row"]) and np.array_equal(sT.cpu().numpy(), ref["s_col"])


def test_mx_nonfinite_rows(lib):
    """A NaN row: scale 0xFF and zero codes in its row blocks and in every column block that meets it."""
    x = make((64, 1056), BF, 4).to(dev)
    x[40, 7] = float("inf")
    q, s, qT, sT, _, _ = lib.mx_layer_norm(x, orientation="dual")
    assert (s[40] == 255).all() and (q[40] == 0).all()
    assert (s[:40] != 255).all() and (s[41:] != 255).all()
    assert (sT[:, 1] == 255).all() and (qT[:, 32:] == 0).all() and (sT[:, 0] != 255).all()
    q, s, _, _, _, _ = lib.mx_layer_norm(x, orientation="row")
    assert (s[40] == 255).all() and (q[40] == 0).all() and (s[39] != 255).all()


def test_mx_feeds_the_product(lib):
    """mx_layer_norm's operand in the MMA layout goes straight into mx_gemm: the
    product of the dequantized operands."""
    x = make((256, 512), BF, 5).to(dev)
    wt = make((256, 512), BF, 6, 0.05).to(dev)
    q, s, _, _, _, _ = lib.mx_layer_norm(x, sf_layout="mma")
    qc, sc, _, _, _, _ = lib.mx_layer_norm(x)
    bq, bs, _, _ = lib.mx_quantize(wt, "e4m3", "row", sf_layout="mma")
    b2, bs2, _, _ = lib.mx_quantize(wt, "e4m3", "row")
    c = lib.mx_gemm(q, s, bq, bs, "e4m3", out_dtype=F32)
    ref = d(lib.mx_dequantize(qc, sc)) @ d(lib.mx_dequantize(b2, bs2)).T
    assert np.abs(d(c) - ref).max() <= 1e-5 * np.abs(ref).max()


# ------------------------------------------------------------------ backward
def backward_ref(dy, x, mean, rstd, w):
    dy, x, mean, rstd = d(dy), d(x), d(mean)[:, None], d(rstd)[:, None]
    n = x.shape[1]
    w = np.ones(n) if w is None else d(w)
    h = (x - mean) * rstd
    g = dy * w
    c1, c2 = g.mean(1, keepdims=True), (g * h).mean(1, keepdims=True)
    dx = rstd * (g - c1 - h * c2)
    k = 28 + n / 1024
    a1, a2 = np.abs(g).mean(1, keepdims=True), np.abs(g * h).mean(1, keepdims=True)
    e_dx = rstd * (4 * U * np.abs(g) + k * U * a1 + np.abs(h) * (k + 6) * U * a2 + 8 * U * (np.abs(c1) + np.abs(h * c2)))
    rows = x.shape[0]
    kr = 100 + rows / 64
    return (dx, (dy * h).sum(0), dy.sum(0), e_dx, (kr + 4) * U * np.abs(dy * h).sum(0) + 1e-40,
            kr * U * np.abs(dy).sum(0) + 1e-40)


def check_backward(lib, dy, x, w):
    _, mean, rstd = lib.layer_norm(x)
    dx, dw, db = lib.layer_norm_backward(dy, x, mean, rstd, w)
    rx, rw, rb, ex, ew, eb = backward_ref(dy, x, mean, rstd, w)
    assert dx.dtype == x.dtype and dw.dtype == db.dtype == F32
    assert (np.abs(d(dx) - rx) <= ex + half_ulp(dx.dtype, rx, ex)).all()
    assert (np.abs(d(dw) - rw) <= ew + U * np.abs(rw)).all()
    assert (np.abs(d(db) - rb) <= eb + U * np.abs(rb)).all()
    again = lib.layer_norm_backward(dy, x, mean, rstd, w)
    assert torch.equal(again[1], dw) and torch.equal(again[2], db) and torch.equal(again[0], dx)
    only, none1, none2 = lib.layer_norm_backward(dy, x, mean, rstd, w, param_grads=False)
    assert torch.equal(only, dx) and none1 is None and none2 is None


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 8), (3, 5), (1, 4096), (2000, 8), (700, 64), (37, 255), (333, 1021),
                                       (64, 1024), (5000, 128), (9, 2049), (13, 4104), (3000, 512), (6, 8192), (3, 8200),
                                       (700, 2048), (2, 14336), (2, 16384), (3, 16385), (2, 20000)])
@pytest.mark.parametrize("xt,dt", [(BF, BF), (F32, F32), (F32, BF), (BF, F32)])
def test_backward_shapes_and_types(lib, rows, cols, xt, dt):
    x = make((rows, cols), xt, rows + cols, 2.0, 0.5).to(dev)
    dy = make((rows, cols), dt, 3, 0.3, 0.05).to(dev)
    w = make((cols,), BF if cols % 2 else F32, 4, 0.3, 1.0).to(dev)
    check_backward(lib, dy, x, w)


@pytest.mark.parametrize("cols,shift", [(1024, 0), (1024, 3), (520, 8)])
def test_backward_strided_rows_and_no_weight(lib, cols, shift):
    wide = make((70, cols + 24), F32, 5).to(dev)
    wdy = make((70, cols + 48), F32, 6).to(dev)
    check_backward(lib, wdy[:, shift:shift + cols], wide[:, shift:shift + cols], None)


def test_backward_of_no_rows_is_zero(lib):
    z = torch.empty(0, 640, device=dev)
    dx, dw, db = lib.layer_norm_backward(z, z, z[:, 0], z[:, 0], torch.ones(640, device=dev))
    assert dx.shape == (0, 640) and (dw == 0).all() and (db == 0).all()


def test_backward_against_differences(lib):
    """Central differences of f(x, w, b) = sum dy * y in float64, step 1e-4:
    the truncation error is of the order 1e-8 of the gradient's scale."""
    rows, cols, step = 3, 72, 1e-4
    x = make((rows, cols), F32, 10)
    w, b = make((cols,), F32, 11, 0.3, 1.0), make((cols,), F32, 12)
    dy = make((rows, cols), F32, 13)
    _, mean, rstd = lib.layer_norm(x.to(dev), w.to(dev), b.to(dev))
    dx, dw, db = lib.layer_norm_backward(dy.to(dev), x.to(dev), mean, rstd, w.to(dev))

    def f(xx, ww, bb):
        m = xx.mean(1, keepdims=True)
        v = ((xx - m) ** 2).mean(1, keepdims=True)
        return float((d(dy) * ((xx - m) / np.sqrt(v + 1e-5) * ww + bb)).sum())

    X, W, B = d(x), d(w), d(b)
    for i, j in [(0, 0), (1, 33), (2, 71)]:
        e = np.zeros_like(X)
        e[i, j] = step
        assert abs((f(X + e, W, B) - f(X - e, W, B)) / (2 * step) - d(dx)[i, j]) < 1e-5
        c = np.zeros_like(W)
        c[j] = step
        assert abs((f(X, W + c, B) - f(X, W - c, B)) / (2 * step) - d(dw)[j]) < 1e-5
        assert abs((f(X, W, B + c) - f(X, W, B - c)) / (2 * step) - d(db)[j]) < 1e-5


def test_backward_nonfinite_rows_stay_alone(lib):
    x, dy = make((6, 512), F32, 14).to(dev), make((6, 512), F32, 15).to(dev)
    _, mean, rstd = lib.layer_norm(x)
    clean = lib.layer_norm_backward(dy, x, mean, rstd)[0]
    dy[2, 100] = float("nan")
    dx, dw, db = lib.layer_norm_backward(dy, x, mean, rstd)
    assert dx[2].isnan().all() and torch.equal(dx[[0, 1, 3, 4, 5]], clean[[0, 1, 3, 4, 5]])
    assert db.isnan().nonzero().flatten().tolist() == [100] and dw.isnan().nonzero().flatten().tolist() == [100]


def test_beyond_2_31_elements(lib):
    """64-bit offsets: 2^31 + elements, sampled rows against the formulas."""
    rows, cols = 131104, 16384
    x = torch.empty(rows, cols, dtype=BF, device=dev)
    g = torch.Generator(device="cuda").manual_seed(1)
    for i in range(0, rows, 8192):
        x[i:i + 8192].normal_(generator=g)
    pick = [0, 65535, 131071, 131072, rows - 1]
    y, mean, rstd = lib.layer_norm(x)
    ry, _, _, ey, _, _ = forward_ref(x[pick], None, None)
    assert (np.abs(d(y[pick]) - ry) <= ey + half_ulp(BF, ry, ey)).all()
    dx, dw, db = lib.layer_norm_backward(y, x, mean, rstd)
    rx, _, _, ex, _, _ = backward_ref(y[pick], x[pick], mean[pick], rstd[pick], None)
    assert (np.abs(d(dx[pick]) - rx) <= ex + half_ulp(BF, rx, ex)).all()
    # y * h sums to the row count (plus rounding of y): every row has taken part
    assert abs(float(dw.double().mean()) / rows - 1) < 1e-2
    del dx, y
    q, s, qT, sT, _, _ = lib.mx_layer_norm(x, orientation="dual")
    for r0 in (0, 131072):
        yy, _, _, e, _, _ = forward_ref(x[r0:r0 + 32], None, None)
        check_blocks(q[r0:r0 + 32].cpu().numpy(), s[r0:r0 + 32].cpu().numpy(), yy, e, "e4m3", omx.FLOOR, "row")
        check_blocks(qT[:, r0:r0 + 32].cpu().numpy(), sT[:, r0 // 32:r0 // 32 + 1].cpu().numpy(), yy.T, e.T, "e4m3",
                     omx.FLOOR, "col")
