"""Layer norm of rows whose deviation is small next to their mean, or nothing.

16-bit rows of up to 16384: the sums of a constant row are exact (11 bits of the number and
13 of their count), and so is the quotient by the width.  Others: the mean is a first sum's,
corrected by the mean of the differences from it.  In a constant row these are all the same
small number of units of the last place, so their sum, and that of their squares, are exact
(below 2^24 units, and units squared), the quotient is the difference itself and the
corrected mean the row's value.  So xh is 0, and with eps = 0 the deviation is 0.

A row of c + (0 or 1), u = 2^-24: what is summed for the mean is, in fp32, the differences
of at most 1 + 27 units of c from a first mean, taken exactly: n u of their mean size, n the
roundings in a row, at most 64 + width / 512; in the shorter fp16 rows, integers below 2^24,
exact.  saved[0] is off by that and its own rounding, half a unit of c.  rstd is off by n u
of itself (the sum of squares, and what is taken from it, is positive) and 4 u (the
hardware's root), xh by the mean's error times rstd, and by (n + 8) u of itself."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
WIDTHS = [1, 2, 3, 7, 8, 15, 30, 41, 56, 104, 120, 240, 328, 480, 768, 776, 1001, 1008, 1600, 2375, 4096, 4097, 6656,
          8191, 8192, 8200, 12344, 16384, 16392, 40001, 300_000]


def _values(dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(6)
    most, lowest = (4.0, 1e-3) if dtype == torch.float16 else (20.0, 1e-12)
    size = torch.exp(torch.rand(120, generator=g, device="cuda") * (math.log(10.0) * most - math.log(lowest)) + math.log(lowest))
    size = size * torch.where(torch.rand(120, generator=g, device="cuda") < 0.5, -1.0, 1.0)
    return torch.cat([torch.tensor([1.0, 1000.0, 1e4, 0.1, 3.0, -3.3, 0.0], device="cuda"), size]).to(dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("width", WIDTHS)
def test_constant_rows(zs, cuda_device, width, dtype):
    value = _values(dtype)
    rows = len(value)
    for offset in (0, 1):
        x = torch.empty(rows * width + offset, dtype=dtype, device="cuda")[offset:].view(rows, width)
        x.copy_(value[:, None].expand(rows, width))
        beta, y = torch.full((width,), 0.5, device="cuda"), torch.empty_like(x)
        saved = torch.empty(rows, 2, device="cuda")
        for eps in (1e-5, 1e-12):
            zs.zero_layer_norm_async(x, None, beta, y, saved=saved, eps=eps)
            assert torch.equal(saved[:, 0], value.float()), value[saved[:, 0] != value.float()][:4]
            assert (y == 0.5).all()
            assert ((saved[:, 1].double() - eps ** -0.5).abs() <= 8 * U * eps ** -0.5).all()
        zs.zero_layer_norm_async(x, None, beta, y, saved=saved, eps=0.0)
        assert (saved[:, 1] == math.inf).all() and y.isnan().all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
@pytest.mark.parametrize("width", [2, 96, 768, 1001, 5000, 8200, 40001])
def test_mean_far_above_the_deviation(zs, cuda_device, width, dtype):
    c = 1e4 if dtype == torch.float32 else 1024.0            # neighbours of it differ by 2^-10, or 1
    x = (c + torch.arange(3 * width, device="cuda") % 2).view(3, width).to(dtype)
    x[2] = c + (torch.rand(width, generator=torch.Generator(device="cuda").manual_seed(width), device="cuda") < 0.1)
    x[2, 0], x[2, 1] = c, c + 1
    y, saved, eps = torch.empty_like(x), torch.empty(3, 2, device="cuda"), 1e-5
    zs.zero_layer_norm_async(x, None, None, y, saved=saved, eps=eps)
    xd = x.double()
    mean = xd.mean(1, keepdim=True)
    rstd = 1.0 / ((xd - mean).square().mean(1, keepdim=True) + eps).sqrt()
    unit, n = 2.0 ** -10, 64 + width / 512                   # of fp32 at both c: 2^13 <= 1e4 < 2^14, and less at 1024
    off_mean = unit / 2 + n * U * (0.5 + 27 * unit)
    assert ((saved[:, :1].double() - mean).abs() <= off_mean).all(), saved[:, :1].double() - mean
    assert ((saved[:, 1:].double() - rstd).abs() <= (n + 4) * U * rstd).all(), saved[:, 1:].double() / rstd - 1
    want = (xd - mean) * rstd
    tol = off_mean * rstd + ((n + 8) * U + HALF[dtype] * 1.01) * want.abs()
    assert ((y.double() - want).abs() <= tol).all(), ((y.double() - want).abs() / tol).max()
