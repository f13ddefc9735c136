"""Rows of very large logits: a vocabulary masked with -1e9 and below in long
runs, rows with nothing else, tops of 1e10, and values around the size at which
the kernel changes the form of its exponent.  Against 64 bits, with the
tolerances that test_gpu_losses.py derives, and for the gradient one more term:
probabilities below 2^-126, the least normal fp32, count as 0, which takes at
most 2^-126 it (|a| + |b| (126 ln 2 + H + 1)) off an element (a and b the
coefficients of logp and H)."""
import math

import pytest
import torch

from test_gpu_losses import HALF_UNIT, TINY, U, _close, _err, _matrix, _policy_inputs, _policy_reference, _reference

pytestmark = pytest.mark.gpu

# (fp16 cannot hold them: it gets there by the temperature alone)
MASKS = [-1e9, -1e10, -1e12, -1e20, -3e35]
CASES = [(t, m, it) for t in (torch.float32, torch.bfloat16) for m in MASKS for it in (0.1, 1.0, 10.0)] + \
        [(torch.float16, -6e4, it) for it in (1.0, 3e4, 1e6)]


def _check(zs, x, y, it):
    """Scoring with and without entropy, and both gradients, of every row."""
    rows, v = x.shape
    f = lambda *n: torch.full(n, math.nan, device="cuda")
    logp, only, ent, saved = f(rows), f(rows), f(rows), f(rows, 2)
    zs.zero_token_logp_async(x, y, logp, entropy=ent, saved=saved, inv_temperature=it)
    zs.zero_token_logp_async(x, y, only, inv_temperature=it)
    z = x.double() * it
    ref_logp, ref_ent, p, lp = _reference(x, y, it, torch.ones(rows, dtype=torch.bool, device="cuda"))
    e = _err(v)
    spread = z.amax(1) - z.gather(1, y[:, None])[:, 0]
    for got in (logp, only):
        _close(got, ref_logp, e + 4 * U * ref_logp.abs() + 3 * U * spread, "logp")
    _close(ent, ref_ent, 4 * e * (1 + ref_ent), "entropy")
    dlogp, dent = torch.linspace(-1, 1.5, rows, device="cuda"), torch.linspace(0.7, -0.9, rows, device="cuda")
    hot = torch.zeros_like(p).scatter_(1, y[:, None], 1.0)
    term = torch.where(p > 0, p * (lp + ref_ent[:, None]), 0.0)
    size = torch.where(p > 0, p * (lp.abs() + ref_ent[:, None] + 1.0), 0.0)
    for with_ent in (False, True):
        out = torch.full((rows, v), 5.0, dtype=x.dtype, device="cuda")
        zs.zero_token_logp_grad_async(x, y, saved, dlogp, out, entropy=ent if with_ent else None,
                                      dentropy=dent if with_ent else None, inv_temperature=it)
        a, b = dlogp.double()[:, None], dent.double()[:, None] if with_ent else 0.0
        want = it * (a * (hot - p) - b * term)
        tol = it * ((2 * e + 300 * U) * (a.abs() * (p + hot) + (4 * b.abs() * size if with_ent else 0.0)))
        flushed = 2.0 ** -126 * it * (a.abs() + (b.abs() * (88.0 + ref_ent[:, None]) if with_ent else 0.0))
        tol = tol + torch.where(p < 2.0 ** -126, flushed, 0.0)
        finite = want.abs() < torch.finfo(x.dtype).max
        _close(out[finite], want[finite], (tol + HALF_UNIT[x.dtype] * want.abs() * 1.01 + TINY[x.dtype])[finite], "dlogits")
        assert not out.isnan().any()


@pytest.mark.parametrize("v", [997, 40_000])
@pytest.mark.parametrize("dtype,mask,it", CASES)
def test_masked_with_large_values(zs, cuda_device, dtype, mask, it, v):
    x, y, g = _matrix(7, v, dtype, 3 + v, spread=2.0 / it)
    x[0, :v - 20] = mask                       # a long run before what is left
    x[1, 20:] = mask                           # and after it
    x[2] = mask                                # nothing else: uniform
    x[3, torch.rand(v, generator=g, device="cuda") < 0.9] = mask
    x[4] = mask
    x[4, v // 3] = 1.0                         # all but one
    x[5, ::2] = mask
    y[0], y[1], y[4], y[5] = v - 3, 4, v // 3, 1
    y[3] = int(torch.nonzero(x[3] != mask)[5])
    x[6] = mask * 1.25 if abs(mask) > 7e4 else mask   # below the others' mask
    _check(zs, x, y, it)


@pytest.mark.parametrize("dtype,top", [(torch.float32, 1e10), (torch.float32, 3e9), (torch.float32, 1e14),
                                       (torch.bfloat16, 1e10), (torch.bfloat16, 1e18), (torch.float32, -1e11)])
@pytest.mark.parametrize("it", [0.1, 1.0, 10.0])
def test_large_tops(zs, cuda_device, dtype, top, it):
    x, y, g = _matrix(4, 2003, dtype, 11)
    x[0, 7], y[0] = top, 7
    x[1, 100:130], y[1] = top, 110
    x[2] = top
    x[3] = top
    x[3, ::2] = top - abs(top) / 64            # far below, at this size
    y[3] = 5
    _check(zs, x, y, it)


@pytest.mark.parametrize("v", [700, 30_011])
@pytest.mark.parametrize("around", [1 << 23, 11_629_080, 1 << 25])
def test_tops_on_both_sides_of_the_change_of_form(zs, cuda_device, around, v):
    """Threads of a row with tops on both sides of 2^24 in units of log2."""
    g = torch.Generator(device="cuda")
    g.manual_seed(v)
    x = torch.randint(-14, 15, (6, v), generator=g, device="cuda").double() + around
    x[3:] = -x[3:]
    x = x.float()
    y = torch.randint(0, v, (6,), generator=g, device="cuda")
    _check(zs, x, y, 1.0)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("mask", [-1e9, -1e10, -1e12, -1e20])
def test_policy_loss_with_a_masked_vocabulary(zs, cuda_device, mask, dtype):
    rows, v = 12, 5003
    hp = dict(clip_low=0.2, clip_high=0.3, dual_clip=2.0, kl_coef=0.1, entropy_coef=0.02)
    x, y, _, _, adv, g = _policy_inputs(rows, v, dtype, 9)
    y %= 100
    x[:, 100:] = mask
    logp64 = torch.log_softmax(x.double(), 1).gather(1, y[:, None])[:, 0]
    old, ref, w = (logp64 - 0.1).float(), (logp64 + 0.2).float(), torch.full((rows,), 1.0 / rows, device="cuda")
    want = _policy_reference(x, y, old, ref, adv, w, hp, torch.ones(rows, dtype=torch.bool, device="cuda"))
    f = lambda *n: torch.full(n, math.nan, device="cuda")
    logp, ent, totals, out = f(rows), f(rows), f(5), torch.empty_like(x)
    zs.zero_policy_loss_async(x, y, old, adv, w, zs.policy(**hp), totals, zs.new_work(), ref_logp=ref, logp=logp,
                              entropy=ent, dlogits=out)
    e = _err(v)
    err = e + 4 * U * want["logp"].abs() + 3 * U * 40
    _close(logp, want["logp"], err, "logp")
    _close(ent, want["entropy"], 4 * e * (1 + want["entropy"]), "entropy")
    _close(out, want["grad"], (2 * err.amax() + 320 * U) * 2 * want["size"] + HALF_UNIT[dtype] * 1.01 * want["grad"].abs() + TINY[dtype], "dlogits")
    slope = adv.double().abs() * 1.3 + 0.1 * 2.3
    tol = (w.double() * ((slope + 1) * (2 * err + 16 * U) + 8 * e * (1 + want["entropy"]))).sum() + U * want["totals"].abs()
    _close(totals, want["totals"], tol, "totals")
