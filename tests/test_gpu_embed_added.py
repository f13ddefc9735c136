"""The embedding's gradient added to an fp32 table: the same bits wherever the table's
rows lie, on 16-byte boundaries, on 8-byte ones or on neither."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


def _place(rows, width, dtype, pad, offset, values):
    buf = torch.full((rows * (width + pad) + offset + 32,), 7.0, dtype=dtype, device="cuda")
    x = buf[offset:offset + rows * (width + pad)].view(rows, width + pad)[:, :width]
    x.copy_(values)
    return x, buf


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("n,vocab,width", [(1, 3, 8), (700, 90, 64), (5000, 40, 24), (3000, 2000, 1032), (20000, 7, 16)])
@pytest.mark.parametrize("size", [1.0, 1e-39])
def test_same_bits_at_every_alignment(zs, cuda_device, n, vocab, width, dtype, size):
    """(size 1e-39: elements and sums that fp32 holds as subnormals)"""
    g = torch.Generator(device="cuda")
    g.manual_seed(n)
    ids = (torch.rand(n, generator=g, device="cuda").square() * vocab).long()
    ids[::7] = vocab                                        # out of range
    dout = torch.randn(n, width, generator=g, device="cuda")
    if size != 1.0:
        dout = torch.zeros_like(dout) if dtype == torch.float16 else dout * size
    start = torch.randn(vocab, width, generator=g, device="cuda") * size
    work = zs.new_embed_work(n, width)
    got = []
    for pad, offset in ((0, 0), (0, 1), (2, 2), (1, 0)):
        src, _ = _place(n, width, dtype, pad, offset, dout)
        table, buf = _place(vocab, width, torch.float32, pad, offset, start)
        zs.zero_embed_grad_async(ids, src, table, work, scale=0.7, accumulate=True)
        got.append(table.clone())
    assert all(torch.equal(t.view(torch.int32), got[0].view(torch.int32)) for t in got[1:])


def test_product_and_sum_are_rounded_by_themselves(zs, cuda_device):
    """One token to an id: sum = dout, so the element is fl(start + fl(dout scale))."""
    n, width, scale = 50, 72, 0.7
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    dout, start = torch.randn(n, width, generator=g, device="cuda"), torch.randn(n, width, generator=g, device="cuda")
    ids = torch.randperm(n, generator=g, device="cuda")
    want = start.clone()
    want[ids] += dout * torch.tensor(scale, device="cuda")
    for pad, offset in ((0, 0), (3, 1)):
        src, _ = _place(n, width, torch.float32, pad, offset, dout)
        table, _ = _place(n, width, torch.float32, pad, offset, start)
        zs.zero_embed_grad_async(ids, src, table, zs.new_embed_work(n, width), scale=scale, accumulate=True)
        assert torch.equal(table, want)


@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("n,vocab,width", [(60, 9, 40), (5000, 30, 24), (5000, 30, 25), (40000, 5, 8)])
def test_nan_and_infinity_stay_in_their_row(zs, cuda_device, n, vocab, width, add, bad):
    g = torch.Generator(device="cuda")
    g.manual_seed(n)
    ids = torch.randint(0, vocab, (n,), generator=g, device="cuda")
    ids[0] = 3
    dout = torch.randn(n, width, generator=g, device="cuda")
    start = torch.randn(vocab, width, generator=g, device="cuda")
    work, out = zs.new_embed_work(n, width), []
    for value in (0.0, bad):
        dout[0, 2] = value
        table = start.clone()
        zs.zero_embed_grad_async(ids, dout, table, work, accumulate=add)
        out.append(table)
    keep = torch.ones(vocab, width, dtype=torch.bool, device="cuda")
    keep[3, 2] = False
    assert torch.equal(out[0][keep], out[1][keep])
    assert out[1][3, 2].isnan() if math.isnan(bad) else out[1][3, 2] == bad
