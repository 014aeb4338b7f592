"""layer_norm at the ends of float32, on each of its kernels."""

import pytest
import torch

pytestmark = pytest.mark.gpu

dev = torch.device("cuda")


def subnormal_rows(rows, cols):
    """Rows of +-sqrt(k) 2^-74.5: mean 0 and variance k 2^-149 exactly, k = 1 .. 64."""
    k = (torch.arange(rows, dtype=torch.float64, device=dev) % 64) + 1
    x = (k.sqrt() * 2.0 ** -74.5).float()[:, None].repeat(1, cols)
    x[:, ::2] *= -1
    return x, k.sqrt().reciprocal() * 2.0 ** 74.5


def many(cols):
    """Enough rows for the kernels that take many, whatever the width."""
    return 81 * torch.cuda.get_device_properties(0).multi_processor_count + 5


@pytest.mark.parametrize("rows,cols", [(70, 1024), (many, 256), (many, 1024), (many, 4096), (many, 1026)])
def test_subnormal_variances(lib, rows, cols):
    """eps 0 and a variance below 2^-126: rstd within 4 float32 roundings, y = +-1 within 8."""
    x, rstd = subnormal_rows(rows(cols) if callable(rows) else rows, cols)
    y, mean, got = lib.layer_norm(x, eps=0.0)
    assert (mean == 0).all()
    assert ((got.double() / rstd - 1).abs() <= 4 * 2.0 ** -24).all()
    assert ((y.double() - x.sign().double()).abs() <= 8 * 2.0 ** -24).all()


@pytest.mark.parametrize("rows,cols,orient", [(64, 512, "row"), (64, 512, "dual"), (64, 4096, "col"), (64, 8192, "dual"),
                                              (64, 8224, "dual")])
def test_subnormal_variances_to_mx(lib, rows, cols, orient):
    x, rstd = subnormal_rows(rows, cols)
    mean, got = lib.mx_layer_norm(x, eps=0.0, orientation=orient)[4:]
    assert (mean == 0).all()
    assert ((got.double() / rstd - 1).abs() <= 4 * 2.0 ** -24).all()
