"""The norm's gradient where numbers are not finite, or leave fp32 on the way: a row's
NaN reaches its own dx and the sums over rows, no other row."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.float16, torch.bfloat16]
HALF = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
U = 2.0 ** -24


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("width", [1, 33, 40, 768, 1001, 5000, 9000])
@pytest.mark.parametrize("where", ["dy", "x"])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_not_finite(zs, cuda_device, width, dtype, where, bad):
    rows, r, k = 21, 13, width // 2
    g = torch.Generator(device="cuda")
    g.manual_seed(width)
    x, dy = (torch.randn(rows, width, generator=g, device="cuda").to(dtype) for _ in range(2))
    gamma = torch.rand(width, generator=g, device="cuda") + 0.5
    y, saved, work = torch.empty_like(x), torch.empty(rows, 2, device="cuda"), zs.new_layer_norm_work(rows, width)
    out = []
    for spoilt in (False, True):
        if spoilt:
            (dy if where == "dy" else x)[r, k] = bad
        zs.zero_layer_norm_async(x, gamma, None, y, saved=saved)
        dx, dgamma, dbeta = torch.empty_like(x), torch.empty(width, device="cuda"), torch.empty(width, device="cuda")
        zs.zero_layer_norm_grad_async(dy, x, gamma, saved, dx, dgamma, dbeta, work)
        out.append((dx, dgamma, dbeta))
    others = torch.arange(rows, device="cuda") != r
    assert torch.equal(out[0][0][others], out[1][0][others]) and not out[1][0][r].isfinite().any()
    columns = torch.arange(width, device="cuda") != k
    if where == "dy":
        assert torch.equal(out[0][1][columns], out[1][1][columns]) and torch.equal(out[0][2][columns], out[1][2][columns])
        assert not out[1][1][k].isfinite() and not out[1][2][k].isfinite()
    else:
        assert out[1][1].isnan().all() and torch.equal(out[0][2], out[1][2])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("width", [5, 20, 33, 40, 1000])
def test_mean_times_rstd_past_fp32(zs, cuda_device, width, dtype):
    """Rows of one large number: xh is 0, so dx = rstd (a - mean a), although mean rstd
    is more than fp32 holds."""
    rows, eps = 9, 1e-12 if width > 100 else 1e-5
    g = torch.Generator(device="cuda")
    g.manual_seed(width)
    value = (3e34 if width > 100 else 5e36)
    x = torch.full((rows, width), value, dtype=dtype, device="cuda")
    dy = torch.randn(rows, width, generator=g, device="cuda").to(dtype)
    gamma = torch.rand(width, generator=g, device="cuda") + 0.5
    saved = torch.stack([x[:, 0].float(), torch.full((rows,), eps ** -0.5, device="cuda")], 1).contiguous()
    assert (saved[:, 0] * saved[:, 1] == math.inf).all()
    dx, dgamma, dbeta = torch.empty_like(x), torch.empty(width, device="cuda"), torch.empty(width, device="cuda")
    zs.zero_layer_norm_grad_async(dy, x, gamma, saved, dx, dgamma, dbeta, zs.new_layer_norm_work(rows, width))
    a, r = dy.double() * gamma.double(), saved[:, 1:].double()
    want = r * (a - a.mean(1, keepdim=True))
    size = r * (a.abs() + a.abs().mean(1, keepdim=True))
    assert ((dx.double() - want).abs() <= (2 * width + 32) * U * size + HALF[dtype] * 1.01 * want.abs()).all()
    assert (dgamma == 0).all() and dbeta.isfinite().all()
