"""Token log-probabilities from hidden states and the vocabulary matrix, and
their gradient, against their definitions in 64 bits.

Tolerances, with u = 2^-24 and D the width.  Products of two 16-bit numbers are
exact in fp32.  A tensor-core instruction adds 16 of them to a sum; taking its
result to be off by at most four units of the last place of the largest number in
it, a sum of n products is off by at most (n / 16 + 1) 8 u A, with A the sum of
the products' magnitudes.
  x      ex = (D / 16 + 1) 8 u A, and 0 where all partial sums are exact (small
         integers over powers of 2)
  ln S   the exponentials (4 u), their arguments (84 u, as in test_gpu_losses.py), the
         sums (V / 256 + 300 terms): E = (400 + V / 128) u, and the logits' ex it
  logp   E + 2 ex it + 4 u |logp| + 4 u |x_y - top| it
  d      relative: half a unit of the type, 2 E + 400 u + 2 ex it of p; in fp16
         also half of its lowest unit, 2^-25, below the largest c at 2^14; and p
         below 2^-126 is 0 (the exponential has no subnormal results): |c| 2^-126
  dH     (sum_j |d_ij w_jk|) (the above + (V / 16 + pieces) 8 u), and half a unit of
         the type of the result;  dW alike over the rows
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float16: 2.0 ** -24, torch.bfloat16: 1e-37}
TYPES = [torch.bfloat16, torch.float16]


def _view(rows, width, dtype, pad, fill=7.0):
    """A matrix inside a larger buffer (rows `pad` elements apart), and the buffer."""
    buf = torch.full((rows + 2, width + pad), fill, dtype=dtype, device="cuda")
    return buf[1:rows + 1, :width], buf


def _around(buf, rows, width):
    """The elements of the buffer outside the matrix."""
    return torch.cat([buf[0], buf[-1], buf[1:rows + 1, width:].reshape(-1)])


def _inputs(rows, vocab, width, dtype, seed, exact=False, pad=0, spread=2.5):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    h, _ = _view(rows, width, dtype, pad)
    w, _ = _view(vocab, width, dtype, pad)
    if exact:      # integers up to 2 times eighths: all sums below 2^24 eighths
        h.copy_(torch.randint(-2, 3, (rows, width), generator=g, device="cuda"))
        w.copy_(torch.randint(-2, 3, (vocab, width), generator=g, device="cuda") / 8.0)
    else:
        h.copy_(torch.randn(rows, width, generator=g, device="cuda"))
        w.copy_(torch.randn(vocab, width, generator=g, device="cuda") * (spread / math.sqrt(width)))
    y = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    return h, w, y, g


def _close(got, want, tol, what):
    got = got.double()
    bad = ~((got - want).abs() <= tol) & ~((got == want) | (got.isnan() & want.isnan()))
    assert not bad.any(), (what, int(bad.sum()), torch.nonzero(bad)[:4].tolist(), got[bad][:4], want[bad][:4])


def _reference(h, w, y, it, valid):
    x = h.double() @ w.double().t()
    size = h.double().abs() @ w.double().abs().t()
    lp = torch.log_softmax(x * it, 1)
    rows = torch.arange(len(y), device="cuda")
    yy = y.clamp(0, w.shape[0] - 1)
    logp = torch.where(valid, lp[rows, yy], 0.0)
    return x, size, lp, logp, yy


def _scratch(zs, rows, width, vocab, gradient, piece=0):
    """Scratch full of NaN, within a larger buffer that has to stay as it is."""
    n = int(zs.lib().zero_head_work_bytes(rows, width, vocab, piece, 1 if gradient else 0))
    assert n > 0
    buf = torch.full((n + 1024,), 255, dtype=torch.uint8, device="cuda")
    return buf[512:512 + n], buf


SHAPES = [(1, 1, 8), (1, 1000, 64), (3, 2, 16), (5, 257, 72), (255, 300, 64), (256, 256, 128), (257, 511, 136),
          (40, 5003, 264), (700, 1031, 96), (9, 50257, 768), (300, 777, 1600), (600, 131, 328), (2, 20000, 4096)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("exact", [True, False])
@pytest.mark.parametrize("rows,vocab,width", SHAPES)
def test_logp_and_gradient(zs, cuda_device, rows, vocab, width, exact, dtype):
    it, pad = 0.75, 0 if width % 16 == 0 else 24
    h, w, y, g = _inputs(rows, vocab, width, dtype, 31 * rows + vocab + width, exact, pad)
    if rows > 2:
        y[1] = -100
        y[-1] = vocab                    # outside the vocabulary: ignored as well
        h[1] = math.nan                  # not used
    valid = (y >= 0) & (y < vocab)
    clean = torch.where(valid[:, None], h, torch.zeros_like(h))
    x, size, lp, ref, yy = _reference(clean, w, y, it, valid)
    e = (400 + vocab / 128) * U
    ex = torch.zeros_like(size) if exact else (width / 16 + 1) * 8 * U * size
    logp, saved = torch.full((rows,), math.nan, device="cuda"), torch.full((rows, 2), math.nan, device="cuda")
    work, buf = _scratch(zs, rows, width, vocab, False)
    zs.zero_head_logp_async(h, w, y, logp, work, saved=saved, inv_temperature=it)
    at = torch.arange(rows, device="cuda")
    xy = x[at, yy]
    tol = e + 2 * ex.amax(1) * it + 4 * U * ref.abs() + 4 * U * (x.amax(1) - xy) * it
    _close(logp, ref, torch.where(valid, tol, 0.0), "logp")
    lse = torch.where(valid, torch.logsumexp(x * it, 1), 0.0)
    _close(saved[:, 0].double() * it + saved[:, 1].double(), lse, torch.where(valid, tol + 4 * U * lse.abs(), 0.0), "saved")
    assert (buf[:512] == 255).all() and (buf[512 + work.numel():] == 255).all()
    alone = torch.empty(rows, device="cuda")
    zs.zero_head_logp_async(h, w, y, alone, work, inv_temperature=it)
    assert torch.equal(alone, logp)

    dlogp = torch.randn(rows, generator=g, device="cuda") / rows
    if rows > 4:
        dlogp[2] = 0.0                   # left out
    live = valid & (dlogp != 0)
    ctrl, scale = zs.new_ctrl(), 256.0
    zs.zero_ctrl_init(ctrl, scale)
    c = torch.where(live, dlogp.double() * (scale * it), 0.0)
    p = lp.exp()
    hot = torch.zeros_like(p)
    hot[at, yy] = 1.0
    d = c[:, None] * (hot - p)
    dd = d.abs() * HALF[dtype] * 1.01 + c.abs()[:, None] * 2.0 ** -126 + c.abs()[:, None] * p * (2 * e + 400 * U + 2 * it * ex.amax(1, keepdim=True))
    if dtype == torch.float16:
        dd += c.abs().max() * 2.0 ** -39
    want_h, want_w = d @ w.double(), d.t() @ clean.double()
    dd_h = dd @ w.double().abs() + (vocab / 16 + 2) * 8 * U * (d.abs() @ w.double().abs())
    dd_w = dd.t() @ clean.double().abs() + (rows / 16 + 2) * 8 * U * (d.abs().t() @ clean.double().abs())
    got = {}
    for piece in (0, 256):
        dh, dh_buf = _view(rows, width, dtype, 16)
        dw, dw_buf = _view(vocab, width, dtype, 8)
        work, buf = _scratch(zs, rows, width, vocab, True, piece)
        zs.zero_head_logp_grad_async(h, w, y, saved, dlogp, dh, dw, work, inv_temperature=it, ctrl_dev=ctrl)
        pieces = 1 if piece == 0 else -(-vocab // piece)
        extra = pieces * 8 * U * (d.abs() @ w.double().abs())
        _close(dh, want_h, (dd_h + extra) * 1.02 + HALF[dtype] * 1.01 * want_h.abs() + TINY[dtype], "dhidden")
        _close(dw, want_w, dd_w * 1.02 + HALF[dtype] * 1.01 * want_w.abs() + TINY[dtype], "dweight")
        assert (dh[~live] == 0).all()
        assert (_around(dh_buf, rows, width) == 7).all() and (_around(dw_buf, vocab, width) == 7).all()
        assert (buf[:512] == 255).all() and (buf[512 + work.numel():] == 255).all()
        got[piece] = (dh, dw)
    assert torch.equal(got[0][1], got[256][1])        # a row of dweight does not depend on the pieces
    # one of the two alone, and the same call again: the same bits
    dh, dw = torch.empty_like(h), torch.empty_like(w)
    zs.zero_head_logp_grad_async(h, w, y, saved, dlogp, dh, None, work, inv_temperature=it, ctrl_dev=ctrl)
    zs.zero_head_logp_grad_async(h, w, y, saved, dlogp, None, dw, work, inv_temperature=it, ctrl_dev=ctrl)
    assert torch.equal(dh, got[256][0]) and torch.equal(dw, got[256][1])


@pytest.mark.parametrize("dtype", TYPES)
def test_saved_of_the_logits_call_serves(zs, cuda_device, dtype):
    """The statistics of zero_token_logp_async on the same logits."""
    rows, vocab, width = 70, 900, 128
    h, w, y, g = _inputs(rows, vocab, width, dtype, 8, exact=True)
    logits = h.float() @ w.float().t()                       # exact
    logp, saved, mine, s2 = (torch.empty(k, device="cuda") for k in (rows, 2 * rows, rows, 2 * rows))
    zs.zero_token_logp_async(logits, y, logp, saved=saved)
    work = zs.new_head_work(rows, width, vocab)
    zs.zero_head_logp_async(h, w, y, mine, work, saved=s2)
    _close(mine, logp.double(), (400 + 900 / 128) * 2 * U + 8 * U * logp.double().abs(), "logp")
    dlogp = torch.randn(rows, generator=g, device="cuda")
    out = []
    for s in (saved, s2):
        dh, dw = torch.empty_like(h), torch.empty_like(w)
        zs.zero_head_logp_grad_async(h, w, y, s, dlogp, dh, dw, work)
        out.append((dh, dw))
    for a, b in zip(*out):
        # d may be rounded to a neighbour: a unit of each product
        assert (a.double() - b.double()).norm() <= 2 * HALF[dtype] * b.double().norm()


@pytest.mark.parametrize("dtype", TYPES)
def test_nothing_left(zs, cuda_device, dtype):
    rows, vocab, width = 300, 700, 64
    h, w, y, _ = _inputs(rows, vocab, width, dtype, 3)
    h[:] = math.nan
    y[:] = -1
    logp, saved = torch.full((rows,), 3.0, device="cuda"), torch.full((rows, 2), 3.0, device="cuda")
    work = _scratch(zs, rows, width, vocab, True)[0]
    zs.zero_head_logp_async(h, w, y, logp, work, saved=saved)
    assert (logp == 0).all() and (saved == 0).all()
    dh, dw = torch.full_like(h, 3.0), torch.full_like(w, 3.0)
    zs.zero_head_logp_grad_async(h, w, y, saved, torch.ones(rows, device="cuda"), dh, dw, work)
    assert (dh == 0).all() and (dw == 0).all()
    # no row at all
    none, dw = h[:0], torch.full_like(w, 3.0)
    zs.zero_head_logp_async(none, w, y[:0], logp[:0], work)
    zs.zero_head_logp_grad_async(none, w, y[:0], saved[:0], logp[:0], torch.empty_like(none), dw, work)
    assert (dw == 0).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_infinities_and_large_logits(zs, cuda_device, dtype):
    rows, vocab, width, inf = 8, 1030, 64, math.inf
    h, w, y, _ = _inputs(rows, vocab, width, dtype, 4, exact=True)
    h.abs_()
    h[:, 0] = 0.0
    h[0] = 0.0
    h[0, 0] = 1.0               # row 0: column 0 of w alone
    w[:, 0] = 0.0
    w[3:, 0] = -inf             # and there all but three entries are impossible
    y[0] = 1
    # (0 times -inf is NaN: every row but 0 and 1 must not meet w's column 0)
    work = zs.new_head_work(rows, width, vocab)
    logp, saved = torch.empty(rows, device="cuda"), torch.empty(rows, 2, device="cuda")
    zs.zero_head_logp_async(h, w, y, logp, work, saved=saved)
    assert abs(float(logp[0]) + math.log(3)) < 1e-6
    assert logp[1:].isnan().all()
    # nothing but -inf; and an impossible label
    w[:, 0] = -inf
    zs.zero_head_logp_async(h[:1], w, y[:1], logp[:1], work, saved=saved[:1])
    assert float(logp[0]) == -inf
    w[5, 0] = 0.0
    zs.zero_head_logp_async(h[:1], w, y[:1], logp[:1], work, saved=saved[:1])
    assert float(logp[0]) == -inf
    # a +inf and a NaN give NaN
    w[:, 0] = 1.0
    w[9, 0] = inf
    zs.zero_head_logp_async(h[:1], w, y[:1], logp[:1], work)
    assert logp[0].isnan()
    w[9, 0] = math.nan
    zs.zero_head_logp_async(h[:1], w, y[:1], logp[:1], work)
    assert logp[0].isnan()
    # logits in the thousands: all mass on the largest
    w[:, 0] = 1.0
    w[700] = 0.0
    w[700, 0] = 4096.0
    y[0] = 700
    zs.zero_head_logp_async(h[:1], w, y[:1], logp[:1], work, saved=saved[:1])
    assert float(logp[0]) == 0.0
    y[0] = 7
    zs.zero_head_logp_async(h[:1], w, y[:1], logp[:1], work, saved=saved[:1])
    assert float(logp[0]) == -4095.0
    dh, dw = torch.empty_like(h[:1]), torch.empty_like(w)
    zs.zero_head_logp_grad_async(h[:1], w, y[:1], saved[:1], torch.ones(1, device="cuda"), dh, dw, work)
    want = w[7].double() - w[700].double()
    assert torch.equal(dh[0].double(), want.to(dtype).double())
    assert torch.equal(dw[7], h[0]) and torch.equal(dw[700], -h[0])
    assert (dw[torch.arange(vocab, device="cuda") % 700 != 7].abs().sum(1)[:5] == 0).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_gradient_of_tiny_and_uneven_weights(zs, cuda_device, dtype):
    """Coefficients around 1e-7 keep their relative accuracy in 16 bits, and rows
    whose coefficients differ by 1e3 stand side by side."""
    rows, vocab, width = 64, 4000, 64
    h, w, y, g = _inputs(rows, vocab, width, dtype, 6)
    work = zs.new_head_work(rows, width, vocab)
    logp, saved = torch.empty(rows, device="cuda"), torch.empty(rows, 2, device="cuda")
    zs.zero_head_logp_async(h, w, y, logp, work, saved=saved)
    ctrl = zs.new_ctrl()
    zs.zero_ctrl_init(ctrl, 65536.0)
    dlogp = torch.where(torch.arange(rows, device="cuda") % 2 == 0, 1e-7, 1e-4) * torch.randn(rows, generator=g, device="cuda")
    dh, dw = torch.empty_like(h), torch.empty_like(w)
    zs.zero_head_logp_grad_async(h, w, y, saved, dlogp, dh, dw, work, ctrl_dev=ctrl)
    d = -torch.softmax(h.double() @ w.double().t(), 1)
    d[torch.arange(rows, device="cuda"), y] += 1.0
    d *= dlogp.double()[:, None] * 65536.0
    want = d @ w.double()
    # per row: half a unit for d, half for the result, and little else
    off = (dh.double() - want).norm(dim=1) / want.norm(dim=1)
    assert (off <= 2.5 * HALF[dtype] + 2.0 ** -24 * 1e3).all(), off.max()
    want = d.t() @ h.double()
    assert (dw.double() - want).norm() <= 2.5 * HALF[dtype] * want.norm()


def test_gradient_against_differences(zs, cuda_device):
    """d sum(dlogp logp) along random directions, by central differences of the forward call in 64 bits."""
    rows, vocab, width = 12, 333, 40
    h, w, y, g = _inputs(rows, vocab, width, torch.float16, 12)
    work = zs.new_head_work(rows, width, vocab)
    logp, saved = torch.empty(rows, device="cuda"), torch.empty(rows, 2, device="cuda")
    zs.zero_head_logp_async(h, w, y, logp, work, saved=saved)
    dlogp = torch.randn(rows, generator=g, device="cuda")
    dh, dw = torch.empty_like(h), torch.empty_like(w)
    zs.zero_head_logp_grad_async(h, w, y, saved, dlogp, dh, dw, work)

    def loss(a, b):
        lp = torch.log_softmax(a @ b.t(), 1)
        return float((lp[torch.arange(rows, device="cuda"), y] * dlogp.double()).sum())

    for _ in range(4):
        u, v = torch.randn(rows, width, generator=g, device="cuda").double(), torch.randn(vocab, width, generator=g, device="cuda").double()
        eps = 1e-5
        slope = (loss(h.double() + eps * u, w.double() + eps * v) - loss(h.double() - eps * u, w.double() - eps * v)) / (2 * eps)
        mine = float((dh.double() * u).sum() + (dw.double() * v).sum())
        size = float((dh.double() * u).abs().sum() + (dw.double() * v).abs().sum())
        assert abs(mine - slope) <= 3 * HALF[torch.float16] * size


@pytest.mark.parametrize("rows", [127, 128, 129, 1023, 1024, 1025, 8192, 8193, 20000])
def test_numbers_of_rows(zs, cuda_device, rows):
    """Around the numbers of rows at which the kernels change, with most rows left out."""
    vocab, width, dtype = 400, 64, torch.bfloat16
    h, w, y, g = _inputs(rows, vocab, width, dtype, rows, exact=True)
    y[torch.rand(rows, generator=g, device="cuda") < 0.7] = -1
    valid = y >= 0
    x, _, lp, ref, yy = _reference(h, w, y, 1.0, valid)
    e = (400 + vocab / 128) * U
    logp, saved = torch.empty(rows, device="cuda"), torch.empty(rows, 2, device="cuda")
    work = zs.new_head_work(rows, width, vocab)
    zs.zero_head_logp_async(h, w, y, logp, work, saved=saved)
    spread = x.amax(1) - x[torch.arange(rows, device="cuda"), yy]
    _close(logp, ref, torch.where(valid, e + 4 * U * ref.abs() + 4 * U * spread, 0.0), "logp")
    dlogp = torch.randn(rows, generator=g, device="cuda") / rows
    dh, dw = torch.empty_like(h), torch.empty_like(w)
    zs.zero_head_logp_grad_async(h, w, y, saved, dlogp, dh, dw, work)
    c = torch.where(valid, dlogp.double(), 0.0)
    d = -lp.exp() * c[:, None]
    d[torch.arange(rows, device="cuda"), yy] += c
    for got, want, size in ((dh, d @ w.double(), d.abs() @ w.double().abs()),
                            (dw, d.t() @ h.double(), d.abs().t() @ h.double().abs())):
        tol = (HALF[dtype] * 1.01 + 2 * e + 400 * U + (rows + vocab) / 2 * U) * size * 1.02 + HALF[dtype] * 1.01 * want.abs() + 1e-30
        _close(got, want, tol, "gradient")
    assert (dh[~valid] == 0).all()


def test_infinite_and_nan_dlogp(zs, cuda_device):
    """One row's coefficient that is no number leaves the other rows' gradients as they are."""
    rows, vocab, width, dtype = 40, 600, 64, torch.float16
    h, w, y, g = _inputs(rows, vocab, width, dtype, 21)
    work = zs.new_head_work(rows, width, vocab)
    logp, saved = torch.empty(rows, device="cuda"), torch.empty(rows, 2, device="cuda")
    zs.zero_head_logp_async(h, w, y, logp, work, saved=saved)
    dlogp = torch.randn(rows, generator=g, device="cuda") * 1e-6
    keep = torch.arange(rows, device="cuda") != 7
    zeroed = dlogp.clone()
    zeroed[7] = 0.0
    want = torch.empty_like(h)
    zs.zero_head_logp_grad_async(h, w, y, saved, zeroed, want, None, work)
    for bad in (math.inf, -math.inf, math.nan):
        dlogp[7] = bad
        dh, dw = torch.empty_like(h), torch.empty_like(w)
        zs.zero_head_logp_grad_async(h, w, y, saved, dlogp, dh, dw, work)
        assert torch.equal(dh[keep], want[keep]) and not dh[7].isfinite().any() and not dw.isfinite().all()


def test_large_offsets(zs, cuda_device):
    """A vocabulary matrix and its gradient of more than 2^32 bytes, rows far apart."""
    rows, vocab, width, stride = 5, 70_001, 64, 32_768
    w = torch.empty(vocab, stride, dtype=torch.bfloat16, device="cuda")[:, :width]
    dw = torch.empty(vocab, stride, dtype=torch.bfloat16, device="cuda")[:, :width]
    h, small, y, g = _inputs(rows, vocab, width, torch.bfloat16, 2, exact=True)
    w.copy_(small)
    y[0] = vocab - 1
    logp, saved, want = (torch.empty(n, device="cuda") for n in (rows, 2 * rows, rows))
    work = zs.new_head_work(rows, width, vocab)
    zs.zero_head_logp_async(h, small, y, want, work, saved=saved)
    zs.zero_head_logp_async(h, w, y, logp, work, saved=saved)
    assert torch.equal(logp, want)
    a, b, c = torch.empty_like(h), torch.empty_like(h), torch.empty_like(small)
    ones = torch.ones(rows, device="cuda")
    zs.zero_head_logp_grad_async(h, small, y, saved, ones, a, c, work)
    zs.zero_head_logp_grad_async(h, w, y, saved, ones, b, dw, work)
    assert torch.equal(a, b) and torch.equal(c, dw)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,vocab,width", [(30, 5003, 264), (200, 9001, 520), (1300, 7000, 64)])
def test_pieces_and_parts(zs, cuda_device, rows, vocab, width, dtype):
    """Pieces of the vocabulary whose sums of dhidden are split into parts as well, the
    last piece shorter: against the whole vocabulary in one piece."""
    h, w, y, g = _inputs(rows, vocab, width, dtype, rows + width)
    logp, saved = torch.empty(rows, device="cuda"), torch.empty(rows, 2, device="cuda")
    whole = zs.new_head_work(rows, width, vocab)
    zs.zero_head_logp_async(h, w, y, logp, whole, saved=saved)
    dlogp = torch.randn(rows, generator=g, device="cuda") / rows
    want_h, want_w = torch.empty_like(h), torch.empty_like(w)
    zs.zero_head_logp_grad_async(h, w, y, saved, dlogp, want_h, want_w, whole)
    d = torch.softmax(h.double() @ w.double().t(), 1) * dlogp.double().abs()[:, None]
    d[torch.arange(rows, device="cuda"), y] += dlogp.double().abs()
    size = d @ w.double().abs()
    for piece in (1024, 2048, 4096, 4352):
        for both in (True, False):
            dh, dw = torch.full_like(h, 7.0), torch.full_like(w, 7.0)
            work, buf = _scratch(zs, rows, width, vocab, True, piece)
            if both:
                zs.zero_head_logp_grad_async(h, w, y, saved, dlogp, dh, dw, work)
            else:
                zs.zero_head_logp_grad_async(h, w, y, saved, dlogp, dh, None, work)
                zs.zero_head_logp_grad_async(h, w, y, saved, dlogp, None, dw, work)
            assert torch.equal(dw, want_w)
            # the same products in another grouping: fp32 sums, then one rounding, perhaps to a neighbour
            tol = (vocab / 16 + 40) * 8 * U * size + 2 * HALF[dtype] * want_h.double().abs() + TINY[dtype]
            _close(dh, want_h.double(), tol, "dhidden")
            assert (buf[:512] == 255).all() and (buf[512 + work.numel():] == 255).all()
