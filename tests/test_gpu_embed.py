"""Embedding lookup and the gradient of its table.

The lookup is one fp32 product and one rounding: exact to the bit.  The gradient
of a token that comes n times is a sum of n terms in fp32, off by at most
(n + 2) u sum|terms| scale, u = 2^-24, plus half a unit of the output's type."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = [torch.float32, torch.float16, torch.bfloat16]
HALF = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 1e-37, torch.float16: 2.0 ** -24, torch.bfloat16: 1e-37}
INT64 = torch.iinfo(torch.int64)


def _place(rows, width, dtype, pad, offset, values=None):
    buf = torch.full((rows * (width + pad) + offset + 32,), 7.0, dtype=dtype, device="cuda")
    x = buf[offset:offset + rows * (width + pad)].view(rows, width + pad)[:, :width]
    if values is not None:
        x.copy_(values)
    return x, buf


def _outside(buf, x):
    keep = torch.ones(buf.numel(), dtype=torch.bool, device="cuda")
    keep.as_strided(x.shape, x.stride(), x.storage_offset())[:] = False
    return buf[keep]


def _ids(kind, n, vocab, g):
    if kind == "one":
        return torch.full((n,), vocab - 1, device="cuda")
    if kind == "each":
        return torch.arange(n, device="cuda").flip(0) % vocab
    if kind == "none":
        return torch.tensor([-1, vocab, INT64.min, INT64.max, 1 << 32], device="cuda").repeat(n // 5 + 1)[:n]
    r = torch.rand(n, generator=g, device="cuda").double()
    ids = ((r * math.log(vocab + 1)).exp().long() - 1).clamp(0, vocab - 1)
    if kind == "skewed":
        return ids
    ids[torch.rand(n, generator=g, device="cuda") < 0.2] = -100          # "holes"
    return ids


SHAPES = [(1, 1, 1, 0, 0), (1, 50257, 768, 0, 0), (8, 3, 7, 0, 1), (100, 40, 33, 5, 3), (1000, 257, 64, 0, 0),
          (1023, 65536, 40, 0, 0), (4097, 1000, 96, 0, 0), (3000, 70000, 130, 2, 1), (20000, 300, 24, 0, 0),
          (5000, 17, 1600, 0, 0), (700, 500, 4100, 0, 0), (40000, 131072, 16, 0, 0), (2, 5, 30000, 0, 0),
          (300_000, 2000, 8, 0, 0), (9000, 900, 512, 8, 8)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,vocab,width,pad,offset", SHAPES)
def test_lookup(zs, cuda_device, n, vocab, width, pad, offset, dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(n + vocab)
    table, _ = _place(vocab, width, dtype, pad, offset)
    table.normal_(generator=g)
    ids = _ids("holes", n, vocab, g)
    if n > 6:
        ids[3], ids[5] = vocab, INT64.max
    inside = (ids >= 0) & (ids < vocab)
    for scale in (1.0, math.sqrt(width), -0.3):
        out, buf = _place(n, width, dtype, pad, offset)
        zs.zero_embed_async(table, ids, out, scale=scale)
        want = (table[ids.clamp(0, vocab - 1)].float() * torch.tensor(scale, dtype=torch.float32, device="cuda")).to(dtype)
        assert torch.equal(out, torch.where(inside[:, None], want, torch.zeros_like(want)))
        assert (_outside(buf, out) == 7).all()
    if n > 1:
        table[0] = math.nan
        ids[0], ids[1] = -1, 0
        zs.zero_embed_async(table, ids, out)
        assert (out[0] == 0).all() and out[1].isnan().all()


@pytest.mark.parametrize("kind", ["skewed", "holes", "one", "each", "none"])
@pytest.mark.parametrize("n,vocab,width,pad,offset", SHAPES)
def test_gradient(zs, cuda_device, n, vocab, width, pad, offset, kind):
    g = torch.Generator(device="cuda")
    g.manual_seed(n + vocab + len(kind))
    ids = _ids(kind, n, vocab, g)
    inside = (ids >= 0) & (ids < vocab)
    rows = ids.clamp(0, vocab - 1)
    scale = 0.7
    need = int(zs.lib().zero_embed_work_bytes(n, width))
    buf = torch.full((need + 512,), 255, dtype=torch.uint8, device="cuda")
    work = buf[256:256 + need]
    count = torch.zeros(vocab, device="cuda").double().index_add_(0, rows, inside.double())
    for dtype, out_dtype, add in ((torch.bfloat16, torch.bfloat16, False), (torch.float16, torch.float32, True),
                                  (torch.float32, torch.float32, False), (torch.bfloat16, torch.bfloat16, True),
                                  (torch.float16, torch.float16, False)):
        dout, _ = _place(n, width, dtype, pad, offset)
        dout.normal_(generator=g)
        dout[~inside] = math.nan                       # not used
        start, _ = _place(vocab, width, out_dtype, pad, offset)
        start.normal_(generator=g)
        dtable, d_buf = _place(vocab, width, out_dtype, pad, offset, start)
        zs.zero_embed_grad_async(ids, dout, dtable, work, scale=scale, accumulate=add)
        src = torch.where(inside[:, None], dout.double(), 0.0)
        zeros = torch.zeros(vocab, width, dtype=torch.float64, device="cuda")
        total, size = zeros.index_add(0, rows, src), zeros.index_add(0, rows, src.abs())
        s32 = float(torch.tensor(scale, dtype=torch.float32))
        want = total * s32 + (start.double() if add else 0.0)
        tol = (count[:, None] + 2) * U * size * s32 + U * want.abs() + HALF[out_dtype] * 1.01 * want.abs() + TINY[out_dtype]
        off = (dtable.double() - want).abs() > tol
        assert not off.any(), (dtype, out_dtype, add, torch.nonzero(off)[:4].tolist(), int(off.sum()))
        if add:
            assert torch.equal(dtable[count == 0], start[count == 0])
        else:
            assert (dtable[count == 0] == 0).all()
        assert (_outside(d_buf, dtable) == 7).all() and (buf[:256] == 255).all() and (buf[256 + need:] == 255).all()
        again, _ = _place(vocab, width, out_dtype, pad, offset, start)
        zs.zero_embed_grad_async(ids, dout, again, work, scale=scale, accumulate=add)
        assert torch.equal(again, dtable)


def test_empty(zs, cuda_device):
    ids, none, dtable = torch.empty(0, dtype=torch.int64, device="cuda"), torch.empty(0, 50, device="cuda"), torch.ones(9, 50, device="cuda")
    zs.zero_embed_async(dtable, ids, none)
    work = zs.new_embed_work(0, 50)
    zs.zero_embed_grad_async(ids, none, dtable, work, accumulate=True)
    assert (dtable == 1).all()
    zs.zero_embed_grad_async(ids, none, dtable, work)
    assert (dtable == 0).all()


def test_gradient_against_differences(zs, cuda_device):
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    ids = torch.randint(0, 12, (60,), generator=g, device="cuda")
    dout, dtable = torch.randn(60, 20, generator=g, device="cuda"), torch.empty(12, 20, device="cuda")
    zs.zero_embed_grad_async(ids, dout, dtable, zs.new_embed_work(60, 20), scale=1.5)
    u = torch.randn(12, 20, generator=g, device="cuda").double()
    # the lookup is linear in the table
    slope = float((u[ids] * 1.5 * dout.double()).sum())
    assert abs(float((dtable.double() * u).sum()) - slope) <= 64 * U * float((u[ids] * 1.5 * dout.double()).abs().sum())


def test_far_rows(zs, cuda_device):
    """Rows of the table more than 2^32 bytes from the first."""
    vocab, width = 70_001, 64
    table = torch.empty(vocab, 32_768, dtype=torch.bfloat16, device="cuda")[:, :width]
    table.normal_()
    ids = torch.tensor([0, vocab - 1, 69_999, 3, vocab - 1], device="cuda")
    out = torch.empty(5, width, dtype=torch.bfloat16, device="cuda")
    zs.zero_embed_async(table, ids, out)
    assert torch.equal(out, table[ids])
    work = zs.new_embed_work(5, width)
    zs.zero_embed_grad_async(ids, out, table, work)
    want = torch.zeros(vocab, width, dtype=torch.bfloat16, device="cuda")
    zs.zero_embed_grad_async(ids, out, want, work)
    assert torch.equal(table, want) and torch.equal(want[3], out[3]) and torch.equal(want[vocab - 1], (out[1].float() * 2).to(torch.bfloat16))


@pytest.mark.parametrize("n", [7, 8, 9, 255, 256, 257, 8191, 8192, 32768, 65535, 65536, 65537])
def test_runs_across_chunks(zs, cuda_device, n):
    """One id from end to end, two that meet anywhere, and one on a chunk's edge: small
    integers, so that every order gives the same sum."""
    width, vocab = 40, 9
    dout = (torch.arange(n, device="cuda")[:, None] * 7 + torch.arange(width, device="cuda")[None]) % 5 - 2
    dout = dout.float()
    work = zs.new_embed_work(n, width)
    for cut in (0, 1, n // 2, n - 1, n // 64 * 64, n // 16 * 16):
        ids = (torch.arange(n, device="cuda") >= cut).long() * 8
        ids = ids[torch.randperm(n, device="cuda")]
        dtable = torch.full((vocab, width), 7.0, device="cuda")
        zs.zero_embed_grad_async(ids, dout, dtable, work)
        want = torch.zeros(vocab, width, device="cuda").double().index_add_(0, ids, dout.double())
        assert torch.equal(dtable.double(), want)
