"""Token log-probabilities, the policy loss and the preference loss against
their definitions in 64 bits, at the shapes and masks where they can go wrong.

Tolerances, with u = 2^-24 the unit of fp32, V the vocabulary:
  ln S    each exponential is off by at most 4 u (two units of the hardware
          exponential) and 3 u |d| of its argument's roundings (|d| <= 40 where
          it counts, in logarithms to the base 2, so 84 u), and a running sum of
          V / 512 + 40 terms by as many u: E = (140 + V / 256) u covers it
  logp    E + 4 u |logp| + 3 u |x_y - top| it
  H       4 E (1 + H): the same errors, weighted by |d|
  dx_i    p_i is off by at most 2 E + 300 u (its own exponent has |q| <= 100),
          times the row's coefficients; plus half a unit of the output type
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = [torch.float32, torch.float16, torch.bfloat16]
HALF_UNIT = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 1e-37, torch.float16: 2.0 ** -24, torch.bfloat16: 1e-37}


def _err(v):
    return (140 + v / 256) * U


def _matrix(rows, vocab, dtype, seed, pad=0, offset=0, spread=3.0):
    """Logits as a view whose rows start `offset` elements into a buffer."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    buf = torch.full((rows * (vocab + pad) + offset + 16,), 7.0, dtype=dtype, device="cuda")
    x = buf[offset:offset + rows * (vocab + pad)].view(rows, vocab + pad)[:, :vocab]
    x.copy_(torch.randn(rows, vocab, generator=g, device="cuda") * spread)
    y = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    return x, y, g


def _reference(x, y, it, valid):
    """logp, entropy, p, ln p in 64 bits; zeros in rows that are not valid."""
    z = x.double() * it
    lp = torch.log_softmax(z, 1)
    p = lp.exp()
    rows = torch.arange(len(y), device="cuda")
    logp = lp[rows, y.clamp(0, x.shape[1] - 1)]
    ent = -torch.where(p > 0, p * lp, 0.0).sum(1)
    zero = torch.zeros((), dtype=torch.float64, device="cuda")
    return torch.where(valid, logp, zero), torch.where(valid, ent, zero), p, lp


def _close(got, want, tol, what):
    got = got.double()
    bad = ~((got - want).abs() <= tol) & ~((got == want) | (got.isnan() & want.isnan()))
    assert not bad.any(), (what, int(bad.sum()), got[bad][:4], want[bad][:4])


def _forward(zs, x, y, it=1.0, **kw):
    n = len(y)
    logp, ent, saved = (torch.full((k,), math.nan, device="cuda") for k in (n, n, 2 * n))
    zs.zero_token_logp_async(x, y, logp, entropy=ent, saved=saved.view(n, 2), inv_temperature=it, **kw)
    return logp, ent, saved.view(n, 2)


SHAPES = [(1, 1, 0, 0), (3, 2, 1, 1), (5, 7, 0, 0), (4, 8, 0, 1), (7, 33, 3, 5), (2, 1000, 0, 0), (9, 4099, 5, 3),
          (3, 50257, 0, 0), (2, 50257, 47, 1), (160, 515, 0, 2), (700, 130, 0, 0), (1, 200_003, 0, 1), (2, 131072, 0, 0),
          (1, 300_000, 0, 0), (2, 900_001, 0, 1)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,vocab,pad,offset", SHAPES)
def test_logp_and_gradient(zs, cuda_device, rows, vocab, pad, offset, dtype):
    x, y, g = _matrix(rows, vocab, dtype, 17 * rows + vocab, pad, offset)
    it = 0.8
    if rows > 2:
        y[1] = -100
        y[-1] = vocab          # outside the vocabulary: ignored as well
        x[1] = math.nan        # not read
    valid = (y >= 0) & (y < vocab)
    logp, ent, saved = _forward(zs, x, y, it)
    ref_logp, ref_ent, p, lp = _reference(x, y, it, valid)
    e = _err(vocab)
    spread = torch.where(valid, (x.double().amax(1) - x.double().gather(1, y.clamp(0, vocab - 1)[:, None])[:, 0]) * it, 0.0)
    _close(logp, ref_logp, e + 4 * U * ref_logp.abs() + 3 * U * spread, "logp")
    _close(ent, ref_ent, 4 * e * (1 + ref_ent), "entropy")
    only = torch.full((rows,), math.nan, device="cuda")
    zs.zero_token_logp_async(x, y, only, inv_temperature=it)      # the variant without entropy
    _close(only, ref_logp, e + 4 * U * ref_logp.abs() + 3 * U * spread, "logp alone")

    dlogp = torch.randn(rows, generator=g, device="cuda")
    dent = torch.randn(rows, generator=g, device="cuda")
    ctrl = zs.new_ctrl()
    zs.zero_ctrl_init(ctrl, 64.0)
    for with_ent in (False, True):
        wide = torch.full((rows, vocab + 9), 5.0, dtype=dtype, device="cuda")
        out = wide[:, 4:4 + vocab]
        zs.zero_token_logp_grad_async(x, y, saved, dlogp, out, entropy=ent if with_ent else None,
                                      dentropy=dent if with_ent else None, inv_temperature=it, ctrl_dev=ctrl)
        a, b = dlogp.double()[:, None], dent.double()[:, None] if with_ent else 0.0
        hot = torch.zeros_like(p).scatter_(1, y.clamp(0, vocab - 1)[:, None], 1.0)
        term = torch.where(p > 0, p * (lp + ref_ent[:, None]), 0.0)
        size = torch.where(p > 0, p * (lp.abs() + ref_ent[:, None] + 1.0), 0.0)
        want = torch.where(valid[:, None], 64.0 * it * (a * (hot - p) - b * term), 0.0)
        tol = 64.0 * it * ((2 * e + 300 * U) * (a.abs() * (p + hot) + (4 * b.abs() * size if with_ent else 0.0)))
        tol = torch.where(valid[:, None], tol, 0.0) + HALF_UNIT[dtype] * want.abs() * 1.01 + TINY[dtype]
        _close(out, want, tol, "dlogits")
        assert (wide[:, :4] == 5).all() and (wide[:, 4 + vocab:] == 5).all(), "written outside the rows"
    # in place: the same bits
    again = x.clone()
    zs.zero_token_logp_grad_async(again, y, saved, dlogp, again, entropy=ent, dentropy=dent, inv_temperature=it,
                                  ctrl_dev=ctrl)
    assert torch.equal(again, out)


@pytest.mark.parametrize("dtype", TYPES)
def test_logp_infinities_and_lowest_values(zs, cuda_device, dtype):
    v, low, inf = 1031, torch.finfo(dtype).min, math.inf
    x, y, _ = _matrix(9, v, dtype, 5)
    x[0, 100:] = -inf                    # a masked vocabulary
    y[0] = 3
    x[1] = -inf                          # nothing left
    x[2] = low                           # a mask of the lowest value everywhere: uniform
    x[3] = low
    x[3, 17] = 1.5                       # and everywhere but once
    y[3] = 17
    x[4, 5] = inf
    x[5, 6] = math.nan
    x[6] = -inf
    x[6, 1000] = 2.0                     # one value left
    y[6] = 1000
    x[7, 9] = -inf                       # the label itself is masked
    y[7] = 9
    x[8] = torch.finfo(dtype).max
    for it in (1.0, 2.5):
        logp, ent, saved = _forward(zs, x, y, it)
        keep = x[0, :100].double() * it
        assert abs(logp[0].item() - torch.log_softmax(keep, 0)[3].item()) <= _err(v) * 4
        assert logp[1].item() == -inf and ent[1].item() == 0.0
        for r in (2, 8):
            assert abs(logp[r].item() + math.log(v)) <= _err(v) and abs(ent[r].item() - math.log(v)) <= 8 * _err(v)
        assert abs(logp[3].item()) <= _err(v) and abs(ent[3].item()) <= _err(v)
        assert math.isnan(logp[4].item()) and math.isnan(logp[5].item()) and math.isnan(ent[4].item())
        assert abs(logp[6].item()) <= _err(v) and abs(ent[6].item()) <= _err(v)
        assert logp[7].item() == -inf and math.isfinite(ent[7].item())
        dlogp, dent = torch.ones(9, device="cuda"), torch.ones(9, device="cuda")
        out = torch.full_like(x, 3.0)
        zs.zero_token_logp_grad_async(x, y, saved, dlogp, out, entropy=ent, dentropy=dent, inv_temperature=it)
        out = out.double()
        assert (out[0, 100:] == 0).all() and (out[1] == 0).all()
        assert out[4].isnan().all() and out[5].isnan().all()
        for r in (0, 2, 3, 6, 7, 8):
            assert out[r].isfinite().all(), r
        assert out[7, 9].item() == pytest.approx(it, rel=2.0 ** -8)


def test_logp_no_rows_other_stream_and_repeats(zs, cuda_device):
    x, y, _ = _matrix(0, 10, torch.float32, 1)
    zs.zero_token_logp_async(x, y, torch.empty(0, device="cuda"))
    x, y, _ = _matrix(37, 9001, torch.bfloat16, 2)
    first = _forward(zs, x, y)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        second = _forward(zs, x, y)
    third = _forward(zs, x, y, stream=s)
    s.synchronize()
    for a, b, c in zip(first, second, third):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_logits_offsets_past_32_bits(zs, cuda_device):
    rows, vocab = 70_001, 32_003                # 2.24e9 elements
    x = torch.empty(rows, vocab, dtype=torch.bfloat16, device="cuda")
    x[:] = torch.linspace(-3, 3, vocab, device="cuda").to(torch.bfloat16)
    y = torch.arange(rows, device="cuda") % vocab
    x[-1] = x[-1].flip(0)
    logp, ent, saved = _forward(zs, x, y)
    lp = torch.log_softmax(x[0].double(), 0)
    e = _err(vocab) + 80 * U
    for r in (0, 1, 32_002, 32_003, 67_108, 70_000):
        want = lp[int(y[r])] if r != 70_000 else lp[vocab - 1 - int(y[r])]
        assert abs(logp[r].item() - want.item()) <= e, r
    keep = [0, 67_108, 70_000]
    zs.zero_token_logp_grad_async(x, y, saved, torch.ones(rows, device="cuda"), x)      # in place
    for r in keep:
        q = lp if r != 70_000 else lp.flip(0)
        want = -q.exp()
        want[int(y[r])] += 1.0
        _close(x[r], want, want.abs() * 2.0 ** -8 + 1e-9, f"row {r}")


# ------------------------------------------------------------------ policy ---

def _policy_inputs(rows, vocab, dtype, seed, pad=0, offset=0):
    x, y, g = _matrix(rows, vocab, dtype, seed, pad, offset)
    logp = torch.log_softmax(x.double(), 1).gather(1, y[:, None])[:, 0]
    noise = torch.randn(rows, generator=g, device="cuda") * 0.3
    for edge in (math.log(0.8), math.log(1.3), math.log(2.0)):     # off the edges of the clipped range
        noise = torch.where((noise - edge).abs() < 1e-3, noise + 3e-3, noise)
    old = (logp - noise).float()
    ref = (logp + torch.randn(rows, generator=g, device="cuda") * 0.3).float()
    adv = torch.randn(rows, generator=g, device="cuda")
    return x, y, old, ref, adv, g


def _policy_reference(x, y, old, ref, adv, w, hp, valid):
    """Per-token loss terms and gradient in 64 bits, by differentiation."""
    rows = torch.nonzero(valid)[:, 0]
    z = x[rows].double().requires_grad_(True)
    lp = torch.log_softmax(z, 1)
    logp = lp.gather(1, y[rows, None])[:, 0]
    safe = lp.masked_fill(lp == -math.inf, 0.0)
    ent = -(lp.exp() * safe).sum(1)
    a = adv[rows].double()
    r = (logp - old[rows].double()).exp()
    held = r.clamp(1 - hp["clip_low"], 1 + hp["clip_high"])
    pg = torch.maximum(-a * r, -a * held)
    cut = -a * r < -a * held
    if hp["dual_clip"]:
        cap = (a < 0) & (pg > -a * hp["dual_clip"])
        pg = torch.where(cap, -a * hp["dual_clip"], pg)
        cut = cut | cap
    kl = torch.zeros_like(pg)
    if ref is not None:
        gap = ref[rows].double() - logp
        kl = gap.exp() - gap - 1
    loss = pg + hp["kl_coef"] * kl - hp["entropy_coef"] * ent
    (loss * w[rows].double()).sum().backward()
    out = {k: torch.zeros(len(y), dtype=torch.float64, device="cuda") for k in ("logp", "entropy", "loss")}
    out["logp"][rows], out["entropy"][rows], out["loss"][rows] = logp.detach(), ent.detach(), loss.detach()
    grad = torch.zeros(x.shape, dtype=torch.float64, device="cuda")
    grad[rows] = z.grad
    out["grad"] = grad
    wr = w[rows].double()
    out["totals"] = torch.stack([(wr * t).sum() for t in (loss.detach(), pg.detach(), kl.detach(), ent.detach(), cut.double())])
    p = lp.detach().exp()
    size = torch.zeros_like(grad)
    hot = torch.zeros_like(p).scatter_(1, y[rows, None], 1.0)
    coef = (a.abs() * r.detach() + hp["kl_coef"] * (1 + (gap.detach().exp() if ref is not None else 0.0)))[:, None]
    size[rows] = wr.abs()[:, None] * (coef * (p + hot) + hp["entropy_coef"] * 4 * p * (safe.detach().abs() + ent.detach()[:, None] + 1))
    out["size"] = size
    return out


POLICIES = [dict(clip_low=0.2, clip_high=0.3, dual_clip=0.0, kl_coef=0.0, entropy_coef=0.0),
            dict(clip_low=0.2, clip_high=0.3, dual_clip=2.0, kl_coef=0.1, entropy_coef=0.02)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("hp", POLICIES, ids=["plain", "all"])
@pytest.mark.parametrize("rows,vocab,pad,offset", [(1, 1, 0, 0), (6, 9, 2, 1), (40, 1003, 0, 3), (5, 50257, 47, 0),
                                                  (900, 260, 0, 0), (2, 200_001, 0, 0), (3, 131072, 0, 0), (2, 450_000, 0, 0), (2, 900_001, 0, 1), (3000, 1500, 0, 0)])
def test_policy_loss(zs, cuda_device, rows, vocab, pad, offset, hp, dtype):
    x, y, old, ref, adv, g = _policy_inputs(rows, vocab, dtype, 3 * rows + vocab, pad, offset)
    ref = ref if hp["kl_coef"] else None
    w = torch.rand(rows, generator=g, device="cuda") / rows
    if rows > 3:
        w[0] = 0.0
        x[0] = math.nan                   # left out: not read
        old[0] = math.nan
        y[2] = -100
    valid = (w != 0) & (y >= 0)
    want = _policy_reference(x, y, old, ref, adv, w, hp, valid)
    f = lambda *n: torch.full(n, math.nan, device="cuda")
    logp, ent, loss, totals, work = f(rows), f(rows) if hp["entropy_coef"] else None, f(rows), f(5), zs.new_work()
    ctrl = zs.new_ctrl()
    zs.zero_ctrl_init(ctrl, 32.0)
    wide = torch.full((rows, vocab + 3), 5.0, dtype=dtype, device="cuda")
    out = wide[:, 1:1 + vocab]

    def call(x, out, **kw):
        zs.zero_policy_loss_async(x, y, old, adv, w, zs.policy(**hp), totals, work, ref_logp=ref, logp=logp,
                                  entropy=ent, token_loss=loss, dlogits=out, ctrl_dev=ctrl, **kw)

    call(x, out)
    e = _err(vocab) + 8 * U * x.double().nan_to_num().abs().amax()
    ratio = torch.where(valid, (want["logp"] - old.double().nan_to_num()).exp(), 0.0)
    err = e + 4 * U * want["logp"].abs()
    _close(logp, want["logp"], err, "logp")
    slope = adv.double().abs() * ratio + hp["kl_coef"] * (1 + (ref.double() - want["logp"]).exp() if ref is not None else 0.0)
    tol = (slope + 1) * (2 * err + 16 * U) + hp["entropy_coef"] * 8 * e * (1 + want["entropy"])
    _close(loss, want["loss"], torch.where(valid, tol, 0.0), "loss")
    if ent is not None:
        _close(ent, want["entropy"], torch.where(valid, 4 * e * (1 + want["entropy"]), 0.0), "entropy")
    else:
        want["totals"][3] = 0.0
    worst = (w.double() * torch.where(valid, tol + 8 * e * (1 + want["entropy"]), 0.0)).sum() + U * want["totals"].abs()
    _close(totals, want["totals"], worst, "totals")
    tol = 32 * (2 * e + 320 * U) * want["size"] * 2 + HALF_UNIT[dtype] * 1.01 * (32 * want["grad"]).abs() + TINY[dtype]
    _close(out, 32 * want["grad"], torch.where(valid[:, None], tol, 0.0), "dlogits")
    assert (wide[:, 0] == 5).all() and (wide[:, 1 + vocab:] == 5).all()
    first = [t.clone() for t in (logp, loss, totals, out)]
    call(x, out)                                           # the scratch is ready again; same bits
    for a, b in zip(first, (logp, loss, totals, out)):
        assert torch.equal(a, b)
    call(x, None)                                          # forward only
    for a, b in zip(first[:3], (logp, loss, totals)):
        _close(b, a.double(), 4 * e * (1 + a.double().abs()) * (1 + slope.max()), "forward only")
    inplace, apart = x.clone(), torch.empty_like(x, memory_format=torch.contiguous_format)
    call(inplace, apart)                                   # (another row alignment than above: its own order of sums)
    call(inplace, inplace)
    assert torch.equal(inplace, apart)


def test_policy_gradient_against_differences(zs, cuda_device):
    """Central differences of the forward loss, step 2^-6 in one logit: the
    truncation is at most h^2 / 6 times a third derivative of some 20 (|A| r
    up to 8, exponentials of order one), 8e-4; the rounding of the losses,
    1e-5 over 2 h, another 3e-4."""
    rows, vocab, h = 24, 61, 2.0 ** -6
    hp = POLICIES[1]
    x, y, old, ref, adv, _ = _policy_inputs(rows, vocab, torch.float32, 77)
    f = lambda *n: torch.empty(*n, device="cuda")
    logp, loss, totals, work, grad = f(rows), f(rows), f(5), zs.new_work(), f(rows, vocab)
    ones = torch.ones(rows, device="cuda")

    def losses(x, out=None):
        zs.zero_policy_loss_async(x, y, old, adv, ones, zs.policy(**hp), totals, work, ref_logp=ref, logp=logp,
                                  token_loss=loss, dlogits=out)
        return loss.double().clone()

    losses(x, grad)
    # rows near an edge of the clipped range have no derivative there
    r = (logp - old).exp()
    clear = ((r - 0.8).abs() > 0.05) & ((r - 1.3).abs() > 0.05) & ((r - 2.0).abs() > 0.08)
    assert clear.sum() > 10
    for i in list(range(0, vocab, 7)):
        e = torch.zeros_like(x)
        e[:, i] = h
        got = (losses(x + e) - losses(x - e)) / (2 * h)
        _close(grad[:, i][clear], got[clear], 1.2e-3, f"logit {i}")
    for r_ in range(rows):                                  # and each row's own label
        e = torch.zeros_like(x)
        e[r_, y[r_]] = h
        got = (losses(x + e)[r_] - losses(x - e)[r_]) / (2 * h)
        if clear[r_]:
            assert abs(got.item() - grad[r_, y[r_]].item()) <= 1.2e-3


def test_policy_nothing_left(zs, cuda_device):
    f = lambda *n: torch.full(n, 9.0, device="cuda")
    work, totals = zs.new_work(), f(5)
    x, y, _ = _matrix(0, 10, torch.float16, 1)
    e = torch.empty(0, device="cuda")
    zs.zero_policy_loss_async(x, y, e, e, None, zs.policy(), totals, work, logp=e)
    assert (totals == 0).all()
    x, y, _ = _matrix(5, 100, torch.float16, 1)
    x[:] = -math.inf
    out, logp, loss, z = torch.full_like(x, 9.0), f(5), f(5), torch.zeros(5, device="cuda")
    zs.zero_policy_loss_async(x, y, z, z + 1, None, zs.policy(kl_coef=1.0), f(5), work, ref_logp=z, logp=logp,
                              token_loss=loss, dlogits=out)
    assert (out == 0).all() and (logp == -math.inf).all() and (loss == 0).all()
    totals = f(5)
    zs.zero_policy_loss_async(x, y, z, z + 1, z, zs.policy(), totals, work, logp=logp, token_loss=loss, dlogits=out)
    assert (totals == 0).all() and (out == 0).all() and (logp == 0).all()


def test_policy_uniform_weights_match_given_ones(zs, cuda_device):
    rows = 12
    x, y, old, ref, adv, _ = _policy_inputs(rows, 77, torch.bfloat16, 4)
    outs = []
    for w in (None, torch.full((rows,), 1.0 / rows, device="cuda")):
        o, t, lp = torch.empty_like(x), torch.empty(5, device="cuda"), torch.empty(rows, device="cuda")
        zs.zero_policy_loss_async(x, y, old, adv, w, zs.policy(), t, zs.new_work(), logp=lp, dlogits=o)
        outs.append((o, t))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


# -------------------------------------------------------------- preference ---

def _pref_reference(logp, ref, mask, cu, w, kind, beta, ls, margin, average):
    ends, pairs = cu.tolist(), (len(cu) - 1) // 2
    leaf = logp.double().nan_to_num(0.0, 0.0, 0.0).requires_grad_(True)
    diff = leaf - (0.0 if ref is None else ref.double().nan_to_num(0.0, 0.0, 0.0))
    scores, sizes = [], []
    for a, b in zip(ends, ends[1:]):
        keep = mask[a:b].bool()
        t = diff[a:b][keep].sum()
        n = max(1, int(keep.sum()))
        scores.append(t / n if average else t)
        sizes.append((logp[a:b][keep].double().abs().sum() + (0 if ref is None else ref[a:b][keep].double().abs().sum())) / (n if average else 1))
    s = torch.stack(scores).view(pairs, 2)
    size = torch.stack(sizes).view(pairs, 2).sum(1)
    h = s[:, 0] - s[:, 1]
    z = beta * h - margin
    sig = torch.nn.functional.logsigmoid
    loss = {"sigmoid": lambda: -(1 - ls) * sig(z) - ls * sig(-z), "hinge": lambda: torch.relu(1 - z),
            "squared": lambda: (h - 0.5 / beta) ** 2}[kind]()
    live = w != 0
    loss = torch.where(live, loss, 0.0)
    (loss * w.double()).sum().backward()
    reward = torch.where(live[:, None], beta * s.detach(), 0.0)
    gain = reward[:, 0] - reward[:, 1]
    totals = torch.stack([(w * t).sum() for t in (loss.detach(), (gain > 0).double(), gain)])
    return loss.detach(), reward.reshape(-1), totals, leaf.grad, size, h.detach()


@pytest.mark.parametrize("kind,ls,margin,average,with_ref", [
    ("sigmoid", 0.0, 0.0, False, True), ("sigmoid", 0.2, 0.4, True, False), ("hinge", 0.0, 0.1, False, True),
    ("squared", 0.0, 0.0, True, True), ("squared", 0.0, 0.0, False, False)])
@pytest.mark.parametrize("pairs,mean,offset", [(1, 1, 0), (1, 5000, 1), (3, 70_000, 2), (17, 40, 0), (700, 9, 3), (40, 1000, 0)])
def test_preference_loss(zs, cuda_device, pairs, mean, offset, kind, ls, margin, average, with_ref):
    g = torch.Generator(device="cuda")
    g.manual_seed(pairs * 31 + mean)
    lens = torch.randint(0, 2 * mean + 1, (2 * pairs,), generator=g, device="cuda")
    if pairs > 2:
        lens[0], lens[1], lens[2] = 0, 1, 0                # empty against one token; empty again
    cu = torch.zeros(2 * pairs + 1, dtype=torch.int64, device="cuda")
    cu[1:] = lens.cumsum(0)
    lead = 5                                               # tokens before the first and after the last sequence
    cu += lead
    n = int(cu[-1]) + 7
    make = lambda: torch.empty(n + offset, device="cuda")[offset:]
    logp, ref = make(), make() if with_ref else None
    logp.copy_(-torch.rand(n, generator=g, device="cuda") * 3)
    if with_ref:
        ref.copy_(logp + torch.randn(n, generator=g, device="cuda") * 0.1)
    mask = torch.rand(n + offset, generator=g, device="cuda")[offset:] < 0.7
    if pairs > 4:
        mask[int(cu[6]):int(cu[7])] = False                # a sequence with nothing left
    logp[~mask] = math.nan                                 # masked: whatever they hold
    if with_ref:
        ref[~mask] = math.inf
    w = torch.rand(pairs, generator=g, device="cuda") / pairs
    if pairs > 4:
        w[4] = 0.0
    beta = 0.1 if with_ref or average else 0.001
    want = _pref_reference(logp, ref, mask, cu, w, kind, beta, ls, margin, average)
    f = lambda k: torch.full((k,), 9.0, device="cuda")
    loss, reward, totals, dlogp, work = f(pairs), f(2 * pairs), f(3), f(n + offset)[offset:], zs.new_work()
    hp = zs.preference(beta, kind, ls, margin, average)

    def call(d):
        zs.zero_preference_loss_async(logp, cu, hp, loss, reward, totals, work, ref_logp=ref, mask=mask, weights=w,
                                      dlogp=d)

    call(dlogp)
    # a difference is off by half a unit of its own, a score by 3 units of the sum of its tokens' sizes
    es = 3 * U * want[4] + U
    slope = beta + 2 * (want[5].abs() + 0.5 / beta) if kind == "squared" else torch.full_like(es, beta)
    _close(loss, want[0], slope * es * 2 + 16 * U * (1 + want[0].abs()) + 4 * U * slope * want[5].abs(), "loss")
    _close(reward, want[1], beta * es.repeat_interleave(2) * 2 + 2 * U * want[1].abs(), "reward")
    tol = (w.double() * (slope * es * 4 + 16 * U * (1 + want[0].abs()) + 4 * U * slope * want[5].abs())).sum() + 4 * U * want[2].abs()
    _close(totals[0::2], want[2][0::2], tol[0::2] if tol.dim() else tol, "totals")
    _close(totals[1:2], want[2][1:2], 4 * U + (w.double() * ((want[1][0::2] - want[1][1::2]).abs() < 4 * beta * es)).sum(), "share")
    inside = torch.zeros(n, dtype=torch.bool, device="cuda")
    inside[int(cu[0]):int(cu[-1])] = True
    assert (dlogp[~inside] == 9).all() and (dlogp[inside & ~mask] == 0).all()
    seq = torch.bucketize(torch.arange(n, device="cuda"), cu[1:], right=True).clamp(max=2 * pairs - 1) // 2
    second = (2.0 if kind == "squared" else beta * beta)   # |d dh / d h| at most
    gtol = ((second * es * 4)[seq] * w.double()[seq] + 24 * U * want[3].abs() + 24 * U * (slope * w.double())[seq])
    live = inside & mask
    if kind == "hinge":                                    # on the edge either side holds
        live &= ((want[5] * beta - margin - 1).abs() > 4 * beta * es + 8 * U)[seq]
    _close(dlogp[live], want[3][live], gtol[live], "dlogp")
    first = [t.clone() for t in (loss, reward, totals, dlogp)]
    call(dlogp)
    for a, b in zip(first, (loss, reward, totals, dlogp)):
        assert torch.equal(a, b)
    call(None)
    for a, b in zip(first[:3], (loss, reward, totals)):
        assert torch.equal(a, b)


def test_preference_gradient_against_differences(zs, cuda_device):
    """Central differences over one pair's first chosen token, step 2^-4: the
    third derivative of the loss is below beta^3, the losses are good to 4e-7,
    so the quotient is good to 1e-5."""
    cu = torch.tensor([0, 3, 9, 14, 20], device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    logp, ref = -torch.rand(20, generator=g, device="cuda"), -torch.rand(20, generator=g, device="cuda")
    f = lambda k: torch.empty(k, device="cuda")
    loss, reward, totals, dlogp, work = f(2), f(4), f(3), f(20), zs.new_work()
    hp = zs.preference(0.3, "sigmoid", 0.1)

    def total(x, d=None):
        zs.zero_preference_loss_async(x, cu, hp, loss, reward, totals, work, ref_logp=ref, dlogp=d)
        return totals[0].item()

    total(logp, dlogp)
    h = 2.0 ** -4
    for i in (0, 2, 5, 9, 13, 19):
        e = torch.zeros(20, device="cuda")
        e[i] = h
        assert abs((total(logp + e) - total(logp - e)) / (2 * h) - dlogp[i].item()) <= 1e-5 + 0.3 ** 3 * h * h


def test_preference_without_pairs_and_offsets_outside(zs, cuda_device):
    f = lambda k: torch.full((k,), 9.0, device="cuda")
    totals, work = f(3), zs.new_work()
    e = torch.empty(0, device="cuda")
    zs.zero_preference_loss_async(e, torch.zeros(1, dtype=torch.int64, device="cuda"), zs.preference(0.1), e, e, totals, work)
    assert (totals == 0).all()
    # no tokens at all: z = -margin
    loss = f(1)
    zs.zero_preference_loss_async(e, torch.zeros(3, dtype=torch.int64, device="cuda"), zs.preference(0.1), loss, f(2), totals, work)
    assert abs(loss.item() - math.log(2)) <= 4 * U
    # offsets past the tokens are cut to them
    x, d = torch.full((8,), -1.0, device="cuda"), f(8)
    cu = torch.tensor([-5, 4, 1 << 40], device="cuda")
    reward = f(2)
    zs.zero_preference_loss_async(x, cu, zs.preference(0.5), loss, reward, totals, work, dlogp=d)
    assert reward.tolist() == [-2.0, -2.0] and abs(loss.item() - math.log(2)) <= 4 * U
    assert d[:4].eq(d[0]).all() and d[4:].eq(-d[0]).all()


# ----------------------------------------------------- together with a step ---

def test_losses_and_step_in_a_graph(zs, cuda_device):
    """Scoring, both losses, their gradients, the norm and the step replayed from
    a CUDA graph give what the calls give."""
    rows, vocab = 48, 3001
    x, y, old, ref, adv, _ = _policy_inputs(rows, vocab, torch.bfloat16, 21)
    f = lambda *n: torch.zeros(*n, device="cuda")
    logp, saved, totals, pair, reward, pref, dlogp = f(rows), f(rows, 2), f(5), f(2), f(4), f(3), f(rows)
    d1, d2 = torch.empty_like(x), torch.empty_like(x)
    cu = torch.tensor([0, 10, 25, 40, rows], device="cuda")
    work, ctrl, sq = zs.new_work(), zs.new_ctrl(), zs.new_sqnorm()
    zs.zero_ctrl_init(ctrl, 4.0)
    master, m, v = f(rows, vocab), f(rows, vocab), f(rows, vocab)
    lst = zs.TensorList([zs.TensorView(d1, master, m, v)])

    def calls():
        zs.zero_token_logp_async(x, y, logp, saved=saved)
        zs.zero_preference_loss_async(logp, cu, zs.preference(0.1), pair, reward, pref, work, ref_logp=ref, dlogp=dlogp)
        zs.zero_token_logp_grad_async(x, y, saved, dlogp, d2, ctrl_dev=ctrl)
        zs.zero_policy_loss_async(x, y, old, adv, None, zs.policy(), totals, work, ref_logp=ref, logp=logp, dlogits=d1,
                                  ctrl_dev=ctrl)
        zs.zero_tensors_sqnorm_async(lst, sq, work, ctrl)
        zs.zero_tensors_adamw_async(lst, zs.adam(1e-3), ctrl, max_norm=1.0, sqnorm_dev=sq)

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        calls()
    s.synchronize()
    want = [t.clone() for t in (logp, pref, dlogp, d1, d2, totals, sq, master, m, v)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for t in (master, m, v, d1, d2, logp, dlogp):
        t.zero_()
    zs.zero_ctrl_init(ctrl, 4.0)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, (logp, pref, dlogp, d1, d2, totals, sq, master, m, v)):
        assert torch.equal(a, b)
    assert zs.read_ctrl(ctrl)["step"] == 1


def test_gradient_that_overflows_its_type_skips_the_step(zs, cuda_device):
    rows, vocab = 8, 500
    x, y, old, ref, adv, _ = _policy_inputs(rows, vocab, torch.float16, 22)
    out, logp, totals, work = torch.empty_like(x), torch.empty(rows, device="cuda"), torch.empty(5, device="cuda"), zs.new_work()
    ctrl, sq = zs.new_ctrl(), zs.new_sqnorm()
    zs.zero_ctrl_init(ctrl, 2.0 ** 24)
    zs.zero_policy_loss_async(x, y, old, adv, None, zs.policy(), totals, work, logp=logp, dlogits=out, ctrl_dev=ctrl)
    assert torch.isinf(out).any() and totals.isfinite().all()
    f = lambda: torch.zeros(rows, vocab, device="cuda")
    master, m, v = f(), f(), f()
    lst = zs.TensorList([zs.TensorView(out, master, m, v)])
    zs.zero_tensors_sqnorm_async(lst, sq, work, ctrl)
    zs.zero_tensors_adamw_async(lst, zs.adam(1e-3), ctrl, max_norm=1.0, sqnorm_dev=sq)
    c = zs.read_ctrl(ctrl)
    assert (c["skipped"], c["step"], c["loss_scale"]) == (1, 0, 2.0 ** 23) and (master == 0).all() and (m == 0).all()
