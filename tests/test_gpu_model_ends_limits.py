"""The head, norm and embedding calls at the ends of their ranges, one size at a time: rows,
vocabulary, width and tokens as large as the header allows, the others small."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
U = 2.0 ** -24


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


@pytest.mark.parametrize("rows,vocab,width", [(1 << 24, 100, 8), (5, 1 << 24, 8), (3, 300, 65536), (200, 300, 65536)])
def test_head(zs, cuda_device, rows, vocab, width):
    """Small integers over powers of 2, so that logits are exact; rows and entries from
    both ends are compared, with the tolerances of test_gpu_head.py."""
    g = _gen(rows + width)
    h = torch.randint(-2, 3, (rows, width), generator=g, device="cuda", dtype=torch.int8).to(BF16)
    w = (torch.randint(-2, 3, (vocab, width), generator=g, device="cuda", dtype=torch.int8) / 8.0).to(BF16)
    if width > 1000:
        w[:, 1000:] = 0.0                       # (logits of a few units)
        w[:, -8:] = 0.125
    y = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    y[0], y[-1] = vocab - 1, 0
    live = torch.rand(rows, generator=g, device="cuda") < 0.9 if rows > 1000 else torch.ones(rows, dtype=torch.bool, device="cuda")
    live[0] = live[-1] = True
    y[~live] = -1
    work = zs.new_head_work(rows, width, vocab, gradient=False)
    logp, saved = torch.empty(rows, device="cuda"), torch.empty(rows, 2, device="cuda")
    zs.zero_head_logp_async(h, w, y, logp, work, saved=saved)
    del work
    at = torch.cat([torch.arange(min(rows, 300), device="cuda"), torch.arange(max(0, rows - 300), rows, device="cuda")]).unique()
    x = h[at].double() @ w.double().t() if vocab < 1 << 20 else torch.cat([h[at].double() @ p.double().t() for p in w.split(1 << 20)], 1)
    lp, pick = torch.log_softmax(x, 1), y[at].clamp(min=0)
    here = torch.arange(len(at), device="cuda")
    e = (400 + vocab / 128) * U
    want = torch.where(live[at], lp[here, pick], 0.0)
    tol = e + 4 * U * want.abs() + 4 * U * (x.amax(1) - x[here, pick])
    assert ((logp[at].double() - want).abs() <= tol).all() and (logp[~live] == 0).all() and logp.isfinite().all()
    dlogp = torch.randn(rows, generator=g, device="cuda")
    dh, dw = torch.full_like(h, 7.0), torch.full_like(w, 7.0)
    zs.zero_head_logp_grad_async(h, w, y, saved, dlogp, dh, dw, zs.new_head_work(rows, width, vocab))
    c = torch.where(live[at], dlogp[at].double(), 0.0)
    d = -lp.exp() * c[:, None]
    d[here, pick] += c
    half = 2.0 ** -8 * 1.01
    dd = d.abs() * half + (c.abs()[:, None] * lp.exp()) * (2 * e + 400 * U) + c.abs()[:, None] * 2.0 ** -126

    def times_w(a, f=lambda t: t):
        return sum(p @ f(q.double()) for p, q in zip(a.split(1 << 20, 1), w.split(1 << 20)))

    want = times_w(d)
    tol = (times_w(dd, torch.abs) + (vocab / 16 + 40) * 8 * U * times_w(d.abs(), torch.abs)) * 1.02 + half * want.abs() + 1e-30
    assert ((dh[at].double() - want).abs() <= tol).all() and (dh[~live] == 0).all()
    if len(at) == rows:
        entries = torch.cat([torch.arange(min(vocab, 300), device="cuda"), torch.arange(max(0, vocab - 300), vocab, device="cuda")]).unique()
        part, size = d[:, entries], h.double().abs()
        want = part.t() @ h.double()
        tol = (dd[:, entries].t() @ size + (rows / 16 + 2) * 8 * U * (part.abs().t() @ size)) * 1.02 + half * want.abs() + 1e-30
        assert ((dw[entries].double() - want).abs() <= tol).all()
    assert dw.isfinite().all() and not (dw == 7.0).all(1).any()


@pytest.mark.parametrize("dtype", [BF16, torch.float32])
def test_widest_norm(zs, cuda_device, dtype):
    """Integers from -2 to 2.  A thread adds 32768 numbers, whose partial sums stay below
    2^11 (8 deviations): each addition is off by at most 2^-14, and so is the mean of the
    differences.  The squares' sum is off by at most n u of itself, n = 32768 and few more."""
    rows, width = 2, 1 << 24
    g = _gen(1)
    x, dy = (torch.randint(-2, 3, (rows, width), generator=g, device="cuda", dtype=torch.int8).to(dtype) for _ in range(2))
    y, saved = torch.empty_like(x), torch.empty(rows, 2, device="cuda")
    zs.zero_layer_norm_async(x, None, None, y, saved=saved)
    mean = x.double().mean(1, keepdim=True)
    rstd = 1.0 / ((x.double() - mean).square().mean(1, keepdim=True) + 1e-5).sqrt()
    off, off_mean = 32800 * U, 2.0 ** -14 * 1.01
    assert ((saved[:, :1].double() - mean).abs() <= off_mean).all() and ((saved[:, 1:] - rstd).abs() <= off * rstd).all()
    half = (U if dtype == torch.float32 else 2.0 ** -8) * 1.01
    want = (x.double() - mean) * rstd
    assert ((y.double() - want).abs() <= (off + half) * want.abs() * 1.01 + off_mean * rstd).all()
    dx, dg, db = torch.empty_like(x), torch.empty(width, device="cuda"), torch.empty(width, device="cuda")
    zs.zero_layer_norm_grad_async(dy, x, None, saved, dx, dg, db, zs.new_layer_norm_work(rows, width))
    a, r = dy.double(), saved[:, 1:].double()
    xh = (x.double() - saved[:, :1].double()) * r
    want = r * (a - a.mean(1, keepdim=True) - xh * (a * xh).mean(1, keepdim=True))
    size = r * (a.abs() + a.abs().mean(1, keepdim=True) + xh.abs() * (a * xh).abs().mean(1, keepdim=True))
    assert ((dx.double() - want).abs() <= 2 * off * size + half * 1.01 * want.abs()).all()
    assert torch.equal(db.double(), a.sum(0)) and ((dg.double() - (a * xh).sum(0)).abs() <= 16 * U * (a * xh).abs().sum(0)).all()


def test_most_norm_rows(zs, cuda_device):
    """2^31 - 1 rows of one element: xh is 0."""
    rows = (1 << 31) - 1
    x = torch.empty(rows, 1, dtype=BF16, device="cuda")
    x.normal_(generator=_gen(2))
    beta, saved = torch.full((1,), 0.5, dtype=BF16, device="cuda"), torch.empty(rows, 2, device="cuda")
    y = torch.empty_like(x)
    zs.zero_layer_norm_async(x, None, beta, y, saved=saved)
    assert (y == 0.5).all() and torch.equal(saved[-1000:, 0], x[-1000:, 0].float()) and torch.equal(saved[:1000, 0], x[:1000, 0].float())
    dg, db = torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
    zs.zero_layer_norm_grad_async(y, x, None, saved, y, dg, db, zs.new_layer_norm_work(rows, 1))
    # (a team's sum of halves stays below 2^24 of them: the sums of blocks round, 35 times in a row)
    assert (y == 0).all() and float(dg) == 0.0 and abs(float(db) / (rows / 2) - 1) <= 40 * U


def test_largest_vocabulary(zs, cuda_device):
    vocab, n, width = 1 << 30, 5000, 1
    g = _gen(3)
    ids = torch.randint(0, vocab, (n,), generator=g, device="cuda")
    ids[:4], ids[4:8] = vocab - 1, 0
    ids[8], ids[9] = vocab, -1
    table = torch.empty(vocab, width, dtype=BF16, device="cuda")
    table.normal_(generator=g)
    out = torch.empty(n, width, dtype=BF16, device="cuda")
    zs.zero_embed_async(table, ids, out)
    inside = (ids >= 0) & (ids < vocab)
    assert torch.equal(out, torch.where(inside[:, None], table[ids.clamp(0, vocab - 1)], 0.0))
    dout = torch.randint(-3, 4, (n, width), generator=g, device="cuda").to(BF16)
    zs.zero_embed_grad_async(ids, dout, table, zs.new_embed_work(n, width))
    real, which = ids[inside].unique(return_inverse=True)
    want = torch.zeros(len(real), width, device="cuda").index_add_(0, which, dout[inside].float())
    assert torch.equal(table[real].float(), want) and int(table.count_nonzero()) == int(want.count_nonzero())


def test_widest_embedding(zs, cuda_device):
    n, vocab, width = 3, 4, 1 << 24
    table = torch.randint(-3, 4, (vocab, width), generator=_gen(4), device="cuda").to(BF16)
    ids, out = torch.tensor([2, 0, 2], device="cuda"), torch.empty(n, width, dtype=BF16, device="cuda")
    zs.zero_embed_async(table, ids, out)
    assert torch.equal(out, table[ids])
    want = torch.zeros(vocab, width, device="cuda").index_add_(0, ids, out.float())
    for dtype, add in ((BF16, False), (torch.float32, True)):
        grad = torch.ones(vocab, width, dtype=dtype, device="cuda")
        zs.zero_embed_grad_async(ids, out, grad, zs.new_embed_work(n, width), accumulate=add)
        assert torch.equal(grad.float(), want + 1 if add else want)


@pytest.mark.parametrize("kind", ["one", "many"])
def test_most_tokens(zs, cuda_device, kind):
    """2^28 tokens; values whose sums are exact: a token in 32 carries 1."""
    n, vocab, width = 1 << 28, 70_000, 1
    ids = torch.full((n,), 5, device="cuda") if kind == "one" else torch.randint(0, vocab, (n,), generator=_gen(5), device="cuda")
    dout = (torch.arange(n, device="cuda", dtype=torch.int32) % 32 == 0).to(BF16)[:, None]
    table = torch.empty(vocab, width, device="cuda")
    zs.zero_embed_grad_async(ids, dout, table, zs.new_embed_work(n, width))
    assert torch.equal(table[:, 0].double(), torch.bincount(ids[::32], minlength=vocab).double())
