"""Layer norm and its gradient against their definitions in 64 bits.

Tolerances, u = 2^-24, D the width, N the rows.  A sum of n fp32 terms, however
grouped, is off by at most n u times the sum of magnitudes; the kernels' groups
make far fewer roundings in a row than n, but n u bounds them all.
  mean   (D + 2) u mean|x|
  rstd   relative: the variance's terms (2 roundings and the mean's error, which
         enters squared and is covered by 2 err_mean dev u^0), (D + 8) u, and 4 u
  y      |xh| and |g| carry those: (D + 16) u |xh g| + |g| rstd err_mean + u |y| + u |b|
  dx     ((2 D + 32) u) rstd (|a| + mean|a| + |xh| mean|a xh|)
  dgamma, dbeta   ((N + 8) u) sum|terms|
and half a unit of the output's type."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = [torch.float32, torch.float16, torch.bfloat16]
HALF = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 1e-37, torch.float16: 2.0 ** -24, torch.bfloat16: 1e-37}


def _place(values, dtype, pad, offset):
    """The values as a matrix whose first element lies `offset` elements into a buffer."""
    rows, width = values.shape
    buf = torch.full((rows * (width + pad) + offset + 32,), 7.0, dtype=dtype, device="cuda")
    x = buf[offset:offset + rows * (width + pad)].view(rows, width + pad)[:, :width]
    x.copy_(values)
    return x, buf


def _close(got, want, tol, what):
    got = got.double()
    bad = ~((got - want).abs() <= tol) & ~((got == want) | (got.isnan() & want.isnan()))
    assert not bad.any(), (what, int(bad.sum()), torch.nonzero(bad)[:4].tolist(), got[bad][:4], want[bad][:4])


def _outside(buf, x):
    keep = torch.ones(buf.numel(), dtype=torch.bool, device="cuda")
    inside = keep.as_strided(x.shape, x.stride(), x.storage_offset())
    inside[:] = False
    return buf[keep]


SHAPES = [(1, 1, 0, 0), (1, 7, 0, 0), (3, 2, 1, 1), (5, 33, 0, 0), (7, 64, 0, 1), (4, 768, 0, 0), (1000, 768, 0, 0),
          (2, 1001, 3, 5), (67, 1600, 0, 0), (9, 4096, 8, 0), (33, 4097, 0, 0), (300, 8, 0, 0), (5000, 24, 0, 0),
          (2, 8192, 0, 0), (3, 12344, 0, 0), (2, 40001, 1, 0), (2, 70000, 0, 0), (1, 300_000, 0, 0), (2500, 128, 0, 0),
          (700, 2048, 0, 0), (150, 5120, 0, 0)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,width,pad,offset", SHAPES)
def test_norm_and_gradient(zs, cuda_device, rows, width, pad, offset, dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(7 * rows + width)
    randn = lambda *n: torch.randn(*n, generator=g, device="cuda")
    params = dtype if rows % 2 else torch.float32
    x, _ = _place(randn(rows, width) * 2.0 + randn(rows, 1), dtype, pad, offset)
    dy, _ = _place(randn(rows, width), dtype, pad, offset)
    gamma, beta, eps = (1.0 + 0.3 * randn(width)).to(params), (0.3 * randn(width)).to(params), 1e-3
    y, y_buf = _place(torch.zeros(rows, width, device="cuda"), dtype, pad, offset)
    saved = torch.full((rows, 2), math.nan, device="cuda")
    zs.zero_layer_norm_async(x, gamma, beta, y, saved=saved, eps=eps)
    xd, gd, bd = x.double(), gamma.double(), beta.double()
    mean = xd.mean(1, keepdim=True)
    rstd = 1.0 / ((xd - mean).square().mean(1, keepdim=True) + eps).sqrt()
    xh = (xd - mean) * rstd
    err_mean = (width + 2) * U * xd.abs().mean(1, keepdim=True)
    err_r = (width + 12) * U + 2 * (err_mean * rstd).square()
    _close(saved[:, :1], mean, err_mean, "mean")
    _close(saved[:, 1:], rstd, err_r * rstd, "rstd")
    want = xh * gd + bd
    tol = ((err_r + 8 * U) * xh.abs() + rstd * err_mean) * gd.abs() + 2 * U * (want.abs() + bd.abs())
    _close(y, want, tol + HALF[dtype] * 1.01 * want.abs() + TINY[dtype], "y")
    assert (_outside(y_buf, y) == 7).all()
    # in place, and without weight and bias
    z = x.clone()
    zs.zero_layer_norm_async(z, gamma, beta, z, eps=eps)
    assert torch.equal(z, y) or pad or offset
    zs.zero_layer_norm_async(x, None, None, z, eps=eps)
    _close(z, xh, (err_r + 8 * U) * xh.abs() + rstd * err_mean + HALF[dtype] * 1.01 * xh.abs() + TINY[dtype], "bare")

    sd = saved.double()
    xh = (xd - sd[:, :1]) * sd[:, 1:]
    a = dy.double() * gd
    m1, m2 = a.mean(1, keepdim=True), (a * xh).mean(1, keepdim=True)
    want = sd[:, 1:] * (a - m1 - xh * m2)
    size = sd[:, 1:] * (a.abs() + a.abs().mean(1, keepdim=True) + xh.abs() * (a * xh).abs().mean(1, keepdim=True))
    dx, dx_buf = _place(torch.zeros(rows, width, device="cuda"), dtype, pad, offset)
    dgamma, dbeta = torch.full_like(gamma, 3.0), torch.full_like(beta, 3.0)
    n = int(zs.lib().zero_layer_norm_work_bytes(rows, width))
    buf = torch.full((n + 512,), 255, dtype=torch.uint8, device="cuda")
    work = buf[256:256 + n]
    zs.zero_layer_norm_grad_async(dy, x, gamma, saved, dx, dgamma, dbeta, work)
    _close(dx, want, (2 * width + 32) * U * size + HALF[dtype] * 1.01 * want.abs() + TINY[dtype], "dx")
    assert (_outside(dx_buf, dx) == 7).all() and (buf[:256] == 255).all() and (buf[256 + n:] == 255).all()
    t = dy.double() * xh
    _close(dgamma, t.sum(0), (rows + 8) * U * t.abs().sum(0) + HALF[params] * 1.01 * t.sum(0).abs() + TINY[params], "dgamma")
    t = dy.double()
    _close(dbeta, t.sum(0), (rows + 8) * U * t.abs().sum(0) + HALF[params] * 1.01 * t.sum(0).abs() + TINY[params], "dbeta")
    # parts of the call, the same call again, dx over dy and over x: the same bits
    only, dg2, db2 = torch.empty_like(dx), torch.empty_like(gamma), torch.empty_like(beta)
    zs.zero_layer_norm_grad_async(dy, x, gamma, saved, only, None, None)
    assert torch.equal(only, dx) or pad or offset
    zs.zero_layer_norm_grad_async(dy, x, gamma, saved, None, dg2, None, work)
    zs.zero_layer_norm_grad_async(dy, x, gamma, saved, None, None, db2, work)
    assert torch.equal(dg2, dgamma) and torch.equal(db2, dbeta)
    keep = dx.clone()
    for place in (dy, x):
        back = place.clone()
        zs.zero_layer_norm_grad_async(dy, x, gamma, saved, place, dg2, db2, work)
        assert torch.equal(place, keep) and torch.equal(dg2, dgamma) and torch.equal(db2, dbeta)
        place.copy_(back)


@pytest.mark.parametrize("width", [96, 768, 5000])
def test_special_rows(zs, cuda_device, width):
    x = torch.randn(6, width, device="cuda")
    x[0] = 3.0                     # constant: xh = 0
    x[1, 5] = math.inf
    x[2, 7] = math.nan
    x[3] = 1e4 + torch.arange(width, device="cuda") % 2      # a mean far above the deviation
    x[4] = 0.0
    beta = torch.full((width,), 0.5, device="cuda")
    y, saved = torch.empty_like(x), torch.empty(6, 2, device="cuda")
    zs.zero_layer_norm_async(x, None, beta, y, saved=saved)
    assert (y[0] == 0.5).all() and (y[4] == 0.5).all() and y[1].isnan().all() and y[2].isnan().all()
    want = torch.nn.functional.layer_norm(x[3].double(), (width,), None, beta.double(), 1e-5)
    assert (y[3].double() - want).abs().max() <= 1e4 * width * U * 4 / 1.0
    assert (y[5].double() - torch.nn.functional.layer_norm(x[5].double(), (width,), None, beta.double(), 1e-5)).abs().max() < 1e-5
    zs.zero_layer_norm_async(x, None, beta, y, eps=0.0)
    assert y[0].isnan().all() and y[5].isfinite().all()


def test_empty(zs, cuda_device):
    x = torch.empty(0, 100, device="cuda")
    zs.zero_layer_norm_async(x, None, None, x)
    dg, db = torch.ones(100, device="cuda"), torch.ones(100, device="cuda")
    zs.zero_layer_norm_grad_async(x, x, None, torch.empty(0, 2, device="cuda"), x, dg, db, zs.new_layer_norm_work(0, 100))
    assert (dg == 0).all() and (db == 0).all()


def test_gradient_against_differences(zs, cuda_device):
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    randn = lambda *n: torch.randn(*n, generator=g, device="cuda")
    x, gamma, beta, dy = randn(20, 77), 1 + 0.2 * randn(77), randn(77), randn(20, 77)
    y, saved = torch.empty_like(x), torch.empty(20, 2, device="cuda")
    zs.zero_layer_norm_async(x, gamma, beta, y, saved=saved)
    dx, dg, db = torch.empty_like(x), torch.empty_like(gamma), torch.empty_like(beta)
    zs.zero_layer_norm_grad_async(dy, x, gamma, saved, dx, dg, db, zs.new_layer_norm_work(20, 77))
    f = lambda a, b, c: float((torch.nn.functional.layer_norm(a, (77,), b, c, 1e-5) * dy.double()).sum())
    for _ in range(4):
        u, v, w, e = randn(20, 77).double(), randn(77).double(), randn(77).double(), 1e-6
        p = (x.double(), gamma.double(), beta.double())
        slope = (f(p[0] + e * u, p[1] + e * v, p[2] + e * w) - f(p[0] - e * u, p[1] - e * v, p[2] - e * w)) / (2 * e)
        parts = [(dx.double() * u), (dg.double() * v), (db.double() * w)]
        size = sum(float(t.abs().sum()) for t in parts)
        # the terms' fp32 errors, and the difference's own (1e-6 in 64 bits)
        assert abs(sum(float(t.sum()) for t in parts) - slope) <= (77 * 4 * U + 1e-6) * size


@pytest.mark.parametrize("x_type", TYPES)
@pytest.mark.parametrize("p_type", TYPES)
@pytest.mark.parametrize("offset", [0, 1])
def test_parameter_types_and_places(zs, cuda_device, x_type, p_type, offset):
    """Every pair of types, parameters on and off a vector boundary, with and without each."""
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    rows, width = 37, 520
    x, dy = (torch.randn(rows, width, generator=g, device="cuda").to(x_type) for _ in range(2))
    gamma, beta, dgamma, dbeta = (torch.randn(width + 1, generator=g, device="cuda").to(p_type)[offset:offset + width] for _ in range(4))
    work = zs.new_layer_norm_work(rows, width)
    xd, m = x.double(), x.double().mean(1, keepdim=True)
    r = 1.0 / ((xd - m).square().mean(1, keepdim=True) + 1e-5).sqrt()
    xh = (xd - m) * r
    y, saved, dx = torch.empty_like(x), torch.empty(rows, 2, device="cuda"), torch.empty_like(x)
    for ga, be in ((gamma, beta), (gamma, None), (None, beta)):
        gd = ga.double() if ga is not None else torch.ones(width, device="cuda").double()
        bd = be.double() if be is not None else torch.zeros(width, device="cuda").double()
        zs.zero_layer_norm_async(x, ga, be, y, saved=saved)
        want = xh * gd + bd
        _close(y, want, 2 * (width + 16) * U * (xh.abs() + 1) * gd.abs() + 2 * U * bd.abs() + HALF[x_type] * 1.01 * want.abs() + TINY[x_type], "y")
        if ga is None:
            continue
        zs.zero_layer_norm_grad_async(dy, x, ga, saved, dx, dgamma, dbeta, work)
        a = dy.double() * gd
        want = r * (a - a.mean(1, keepdim=True) - xh * (a * xh).mean(1, keepdim=True))
        size = r * (a.abs() + a.abs().mean(1, keepdim=True) + xh.abs() * (a * xh).abs().mean(1, keepdim=True))
        _close(dx, want, (4 * width + 64) * U * size + HALF[x_type] * 1.01 * want.abs() + TINY[x_type], "dx")
        for got, t in ((dgamma, dy.double() * xh), (dbeta, dy.double())):
            _close(got, t.sum(0), (2 * width + rows + 64) * U * (t.abs() + dy.double().abs()).sum(0) + HALF[p_type] * 1.01 * t.sum(0).abs() + TINY[p_type], "params")


def test_far_rows(zs, cuda_device):
    """Rows more than 2^32 bytes from the first."""
    x = torch.empty(70_000, 32_768, dtype=torch.bfloat16, device="cuda")[:, :64]
    x.normal_()
    y, want = torch.empty_like(x), torch.empty(70_000, 64, dtype=torch.bfloat16, device="cuda")
    zs.zero_layer_norm_async(x.contiguous(), None, None, want)
    zs.zero_layer_norm_async(x, None, None, y)
    assert torch.equal(y, want)
