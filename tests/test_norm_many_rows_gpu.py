"""The kernels that the layer norms take for many rows: rings of whole rows
(forward, backward) and clusters that walk over tiles (to MX).

Row counts come from the SM count: above what makes every group of threads of
a ring take several rows, and every cluster several tiles.  Formulas and
tolerances are those of the other layer-norm tests: the rings' sums have no
more roundings than they allow (a thread's 64 bytes in pairs and a tree, five
over lanes, five over warps; a column sum a group's rows, at most 16 groups
and 152 parts in a tree)."""

import pytest
import torch

from oracle import mx as omx
from tests.test_norm_gpu import check_backward, check_blocks, check_forward, d, forward_ref, make

pytestmark = pytest.mark.gpu

dev = torch.device("cuda")
BF, F32 = torch.bfloat16, torch.float32
TYPES = [(BF, BF), (F32, F32), (F32, BF), (BF, F32)]


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def rows_for(cols, elems, threads, each):
    """``each`` rows for every group of a CTA on each SM, when a thread holds ``elems`` elements, and three more."""
    g = -(-cols // (32 * elems)) * 32
    return each * max(1, min(15 if g > 32 else 32, threads // g)) * sms() + 3


def padded(rows, cols, dtype, seed, pad, shift, **kw):
    """[rows][cols] with ``pad`` further elements between rows, ``shift`` of them before the first."""
    wide = make((rows, cols + pad), dtype, seed, **kw).to(dev)
    return wide[:, shift:shift + cols]


def params(cols, kinds, seed):
    return [None if k is None else make((cols,), k, seed + i, 0.3, 1.0 - i).to(dev) for i, k in enumerate(kinds)]


@pytest.mark.parametrize("cols", [256, 264, 1024, 2056, 4096, 14336, 14344])
@pytest.mark.parametrize("xt,yt", TYPES)
@pytest.mark.parametrize("kinds", [(BF, BF), (F32, BF)])
def test_forward_ring(lib, cols, xt, yt, kinds):
    """One to many warps a row, whole and partial rows, weights of both types in shared memory."""
    rows = rows_for(cols, 64 // (4 if xt == F32 else 2), 640, 4)
    x = make((rows, cols), xt, cols, 2.0, 0.5).to(dev)
    check_forward(lib, x, *params(cols, kinds, 1), yt)


@pytest.mark.parametrize("kinds", [(None, None), (BF, None), (None, BF), (F32, None), (None, F32)])
@pytest.mark.parametrize("xt", [BF, F32])
def test_forward_ring_without_weight_or_bias(lib, xt, kinds):
    rows = rows_for(1032, 16, 640, 4)
    check_forward(lib, make((rows, 1032), xt, 5).to(dev), *params(1032, kinds, 6))


@pytest.mark.parametrize("cols,pad,shift", [(257, 0, 0), (1021, 0, 0), (1022, 2, 1), (1023, 6, 3), (2049, 9, 8), (5001, 0, 0),
                                            (512, 8, 8), (512, 5, 2), (1028, 4, 4)])
@pytest.mark.parametrize("xt,yt", TYPES)
def test_forward_ring_odd_widths_and_strides(lib, cols, pad, shift, xt, yt):
    """Rows that start and end inside 16-byte words, and strided rows that do not."""
    rows = max(rows_for(cols, 16, 640, 4), rows_for(cols, 32, 640, 4))
    x = padded(rows, cols, xt, cols + shift, pad, shift, scale=2.0, offset=0.5)
    check_forward(lib, x, *params(cols, (F32, BF), 2), yt)


@pytest.mark.parametrize("cols", [1024, 1026, 4104])
def test_forward_ring_undefined_rows_stay_alone(lib, cols):
    rows = rows_for(cols, 16, 640, 5)
    x = make((rows, cols), F32, 8).to(dev)
    clean = lib.layer_norm(x)
    bad = [0, 1, rows // 3, rows // 2, rows - 1]
    for i, r in enumerate(bad):
        x[r, (i * 311) % cols] = float("nan") if i % 2 else float("inf")
    got = lib.layer_norm(x)
    keep = torch.ones(rows, dtype=torch.bool, device=dev)
    keep[bad] = False
    assert got[0][bad].isnan().all()
    for a, b in zip(got, clean):
        assert torch.equal(a[keep], b[keep])


@pytest.mark.parametrize("cols", [128, 136, 1024, 1032, 4096, 4104, 8192, 8200, 16384])
@pytest.mark.parametrize("xt,dt", TYPES)
def test_backward_ring(lib, cols, xt, dt):
    """One to many warps a row, whole and partial, rows that stay in registers
    and rows that are read twice (more than 16 elements a thread)."""
    rows = rows_for(cols, 16, 512, 3)
    x = make((rows, cols), xt, cols, 2.0, 0.5).to(dev)
    dy = make((rows, cols), dt, 3, 0.3, 0.05).to(dev)
    check_backward(lib, dy, x, params(cols, (BF if cols % 256 else F32,), 4)[0])


@pytest.mark.parametrize("cols,pad,shift", [(129, 0, 0), (1021, 0, 0), (1022, 3, 1), (2049, 7, 5), (4099, 0, 0), (8191, 1, 1),
                                            (8195, 0, 0), (512, 8, 8)])
@pytest.mark.parametrize("xt,dt", TYPES)
def test_backward_ring_odd_widths_and_strides(lib, cols, pad, shift, xt, dt):
    rows = rows_for(cols, 16, 512, 3)
    x = padded(rows, cols, xt, cols, pad, shift, scale=2.0, offset=0.5)
    dy = padded(rows, cols, dt, 3, 2 * pad, shift, scale=0.3)
    check_backward(lib, dy, x, params(cols, (F32 if cols % 3 else BF,), 4)[0])


@pytest.mark.parametrize("cols", [1024, 8200, 1021])
def test_backward_ring_undefined_rows_and_no_weight(lib, cols):
    rows = rows_for(cols, 16, 512, 4)
    x, dy = make((rows, cols), BF, 14).to(dev), make((rows, cols), BF, 15).to(dev)
    _, mean, rstd = lib.layer_norm(x)
    clean = lib.layer_norm_backward(dy, x, mean, rstd)[0]
    check_backward(lib, dy, x, None)
    bad = [0, rows // 2, rows - 1]
    for r in bad:
        dy[r, 100] = float("nan")
    dx, dw, db = lib.layer_norm_backward(dy, x, mean, rstd)
    keep = torch.ones(rows, dtype=torch.bool, device=dev)
    keep[bad] = False
    assert dx[bad].isnan().all() and torch.equal(dx[keep], clean[keep])
    for s in (dw, db):
        assert s.isnan().nonzero().flatten().tolist() == [100]


# ------------------------------------------------------------------ to MX: several tiles of 32 rows to a cluster
def slices(out, rows, cols, r0, n, sf):
    """The part of mx_layer_norm's outputs that belongs to rows [r0, r0 + n)."""
    q, s, qT, sT, mean, rstd = out
    per = qT.shape[1] * 32 // rows          # bytes of 32 rows in a row of the column copy
    parts = [q[r0:r0 + n], qT[:, r0 // 32 * per:(r0 + n) // 32 * per], mean[r0:r0 + n], rstd[r0:r0 + n]]
    if sf == "canonical":
        parts += [s[r0:r0 + n], sT[:, r0 // 32:(r0 + n) // 32]]
    else:                                   # 512-byte chunks of 128 rows and four blocks
        parts += [s.reshape(-1)[r0 * cols // 32:(r0 + n) * cols // 32],
                  sT.reshape(cols // 128, rows // 128, 512)[:, r0 // 128:(r0 + n) // 128]]
    return [p.reshape(-1) for p in parts]


@pytest.mark.parametrize("cols,xt,fmt,sf,tail", [
    (512, BF, "e4m3", "mma", 0), (1056, BF, "e5m2", "canonical", 32), (1024, F32, "e4m3", "mma", 0),
    (4096, BF, "e4m3", "mma", 0), (4000, BF, "e2m1", "canonical", 96), (4096, F32, "e2m1", "mma", 0),
    (4096, BF, "e4m3", "canonical", 0), (8192, BF, "e4m3", "mma", 0), (6016, F32, "e5m2", "mma", 0),
    (8192, F32, "e4m3", "canonical", 64), (8320, BF, "e4m3", "mma", 0), (12288, F32, "e2m1", "canonical", 32)])
@pytest.mark.parametrize("mode", ["floor", "ceil"])
def test_mx_many_tiles(lib, cols, xt, fmt, sf, tail, mode):
    """Five tiles or more to a cluster: every byte is that of a call on 128 rows
    (one tile to a cluster), and sampled tiles hold the blocks of y."""
    slabs = -(-cols // (1024 if 4096 < cols <= 8192 else 512))
    rows = max(5 * 32 * -(-2 * sms() // slabs), 1280) // 128 * 128 + 128 + tail
    x = make((rows, cols), xt, cols, 2.0, 0.3).to(dev)
    x[:, 5] *= 30
    w, b = params(cols, (F32, BF), 1)
    out = lib.mx_layer_norm(x, w, b, 1e-5, fmt, "dual", mode, sf)
    for r0 in range(0, rows, 128):
        n = min(128, rows - r0)
        small = lib.mx_layer_norm(x[r0:r0 + n], w, b, 1e-5, fmt, "dual", mode, sf)
        for got, want in zip(slices(out, rows, cols, r0, n, sf), slices(small, n, cols, 0, n, sf)):
            assert torch.equal(got, want), r0
    only = lib.mx_layer_norm(x, w, b, 1e-5, fmt, "col", mode, sf)
    assert only[0] is None and all(torch.equal(p, r) for p, r in zip(only[2:], out[2:]))
    m = {"floor": omx.FLOOR, "ceil": omx.CEIL}[mode]
    for r0 in (0, rows // 3 // 128 * 128, (rows - 32) // 128 * 128):
        n = min(128, rows - r0)
        y, rm, rr, ey, em, er = forward_ref(x[r0:r0 + n], w, b)
        q, qT, mean, rstd, s, sT = slices(out, rows, cols, r0, n, sf)
        assert (abs(d(mean) - rm) <= em + 2.0 ** -24 * abs(rm)).all() and (abs(d(rstd) - rr) <= er).all()
        for qq, ss, yy, e in ((q, s, y, ey), (qT, sT, y.T, ey.T)):
            ss = ss.cpu().numpy().reshape(yy.shape[0], yy.shape[1] // 32)
            if sf == "mma":
                ss = omx.sf_from_mma(ss, yy.shape[0], yy.shape[1] // 32)
            check_blocks(qq.cpu().numpy().reshape(yy.shape[0], -1), ss, yy, e, fmt, m, r0)


def test_mx_many_tiles_with_undefined_rows(lib):
    """A NaN row in a tile of the middle: its row blocks and the column blocks of its 32 rows alone."""
    cols = 4096
    rows = 5 * 32 * -(-2 * sms() // 8) // 128 * 128 + 128
    x = make((rows, cols), BF, 9).to(dev)
    clean = lib.mx_layer_norm(x, orientation="dual")
    bad = rows // 64 * 32 + 7
    x[bad, 1234] = float("nan")
    q, s, qT, sT, _, _ = lib.mx_layer_norm(x, orientation="dual")
    keep = torch.arange(rows, device=dev) != bad
    assert (q[bad] == 0).all() and (s[bad] == 255).all()
    assert torch.equal(q[keep], clean[0][keep]) and torch.equal(s[keep], clean[1][keep])
    t = bad // 32
    assert (qT[:, 32 * t:32 * t + 32] == 0).all() and (sT[:, t] == 255).all()
    tiles = torch.arange(rows // 32, device=dev) != t
    assert torch.equal(sT[:, tiles], clean[3][:, tiles])
    assert torch.equal(qT.view(cols, -1, 32)[:, tiles], clean[2].view(cols, -1, 32)[:, tiles])
