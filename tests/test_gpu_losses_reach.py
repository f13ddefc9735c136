"""Parts of the loss kernels that only many rows, many rows left out or certain
alignments reach: a cluster's second batch of rows, the dealing of live rows
where most are dead, and the preference loss's vectors where the buffers' common
boundary lies one to three tokens in.  Tolerances as in test_gpu_losses.py."""
import math

import pytest
import torch

from test_gpu_losses import HALF_UNIT, TINY, U, _close, _err, _pref_reference

pytestmark = pytest.mark.gpu

CHUNK = 1 << 25                # logits of a piece of the reference


def _dead(rows, how, g):
    """Which rows are left out."""
    i = torch.arange(rows, device="cuda")
    if how == "one left":
        return i != rows * 2 // 3
    if how == "runs":
        return (i // 97) % 3 != 1
    if how == "none":
        return i < 0
    return torch.rand(rows, generator=g, device="cuda") < how


def _check_rows(zs, rows, vocab, how, dtype=torch.bfloat16, seed=1):
    """Scoring, its gradient and the policy loss with its gradient against 64 bits."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.empty(rows, vocab, dtype=dtype, device="cuda")
    step = max(1, CHUNK // vocab)
    for a in range(0, rows, step):
        x[a:a + step] = (torch.randn(min(step, rows - a), vocab, generator=g, device="cuda") * 3).to(dtype)
    y = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    dead = _dead(rows, how, g)
    labels = torch.where(dead, torch.full_like(y, -100), y)
    f = lambda *n: torch.full(n, math.nan, device="cuda")
    logp, saved, grad = f(rows), f(rows, 2), torch.full_like(x, math.nan)
    zs.zero_token_logp_async(x, labels, logp, saved=saved)
    dlogp = torch.randn(rows, generator=g, device="cuda")
    zs.zero_token_logp_grad_async(x, labels, saved, dlogp, grad)
    # advantages of one sign and a ratio of 1: loss = -A, dlogp = -A w
    w = torch.where(dead, 0.0, 1.0 / rows)
    adv = torch.rand(rows, generator=g, device="cuda") + 0.5
    plp, loss, totals, pgrad = f(rows), f(rows), f(5), torch.full_like(x, math.nan)
    old = torch.where(dead, math.nan, logp)
    zs.zero_policy_loss_async(x, y, old, adv, w, zs.policy(), totals, zs.new_work(), logp=plp, token_loss=loss, dlogits=pgrad)
    e = _err(vocab)
    total = 0.0
    for a in range(0, rows, step):
        b, live = min(rows, a + step), ~dead[a:a + step]
        lp = torch.log_softmax(x[a:b].double(), 1)
        want = torch.where(live, lp.gather(1, y[a:b, None])[:, 0], 0.0)
        tol = torch.where(live, e + 4 * U * want.abs() + 3 * U * 40, 0.0)
        _close(logp[a:b], want, tol, f"logp from row {a}")
        _close(plp[a:b], want, tol, f"policy logp from row {a}")
        err = 2 * tol + 16 * U
        ratio = torch.where(live, (want - old[a:b].double().nan_to_num()).exp(), 0.0)
        wl = torch.where(live, -adv[a:b].double() * ratio, 0.0)
        _close(loss[a:b], wl, torch.where(live, adv[a:b].double() * err * 2, 0.0), f"loss from row {a}")
        total += (w[a:b].double() * wl).sum().item()
        p = lp.exp()
        hot = torch.zeros_like(p).scatter_(1, y[a:b, None], 1.0)
        for got, c in ((grad, dlogp.double()), (pgrad, -adv.double() * w.double())):
            c = torch.where(live, c[a:b], 0.0)[:, None]
            wg = c * (hot - p)
            # (the policy's coefficient carries the ratio's error as well)
            tg = c.abs() * (p + hot) * (2 * e + 300 * U + err[:, None]) + HALF_UNIT[dtype] * wg.abs() * 1.01
            _close(got[a:b], wg, torch.where(live[:, None], tg + TINY[dtype], 0.0), f"dlogits from row {a}")
        del lp, p, hot
    assert abs(totals[0].item() - total) <= (2 * e + 200 * U) * 3 + U * abs(total)


@pytest.mark.parametrize("rows,vocab", [(400_003, 130), (170_001, 8200)])
@pytest.mark.parametrize("how", ["none", 0.3, 0.9])
def test_more_rows_than_the_clusters_take_at_a_time(zs, cuda_device, rows, vocab, how):
    _check_rows(zs, rows, vocab, how)


@pytest.mark.parametrize("rows,vocab", [(5003, 1501), (2100, 12_007), (1300, 70_000)])
@pytest.mark.parametrize("how", [0.3, 0.6, 0.9, 0.99, "runs", "one left"])
@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_most_rows_left_out(zs, cuda_device, rows, vocab, how, dtype):
    _check_rows(zs, rows, vocab, how, dtype)


@pytest.mark.parametrize("kind,average,with_ref", [("sigmoid", False, True), ("hinge", True, True), ("squared", True, False)])
@pytest.mark.parametrize("pairs,mean", [(1, 6), (1, 9000), (40, 5), (300, 70), (9, 3000)])
@pytest.mark.parametrize("offset", [0, 1, 2, 3])
def test_preference_vectors_off_the_buffers_start(zs, cuda_device, pairs, mean, offset, kind, average, with_ref):
    """Every buffer `offset` elements past a boundary of four: the mask's bytes
    and the floats have theirs at the same token."""
    g = torch.Generator(device="cuda")
    g.manual_seed(7 * pairs + mean)
    lens = torch.randint(0, 2 * mean + 1, (2 * pairs,), generator=g, device="cuda")
    cu = torch.zeros(2 * pairs + 1, dtype=torch.int64, device="cuda")
    cu[1:] = lens.cumsum(0)
    cu += 2
    n = int(cu[-1]) + 3
    part = lambda dtype: torch.zeros(n + offset + 4, dtype=dtype, device="cuda")[offset:offset + n]
    logp, ref, mask, dlogp = part(torch.float32), part(torch.float32), part(torch.bool), part(torch.float32)
    logp.copy_(-torch.rand(n, generator=g, device="cuda") * 3)
    ref.copy_(logp + torch.randn(n, generator=g, device="cuda") * 0.1)
    mask.copy_(torch.rand(n, generator=g, device="cuda") < 0.7)
    assert all(t.data_ptr() % (4 * t.element_size()) == offset * t.element_size() for t in (logp, ref, mask, dlogp))
    dlogp.fill_(9.0)
    logp[~mask] = math.nan
    w = torch.rand(pairs, generator=g, device="cuda") / pairs
    beta = 0.1
    f = lambda k: torch.full((k,), 9.0, device="cuda")
    loss, reward, totals = f(pairs), f(2 * pairs), f(3)
    zs.zero_preference_loss_async(logp, cu, zs.preference(beta, kind, average=average), loss, reward, totals, zs.new_work(),
                                  ref_logp=ref if with_ref else None, mask=mask, weights=w, dlogp=dlogp)
    want = _pref_reference(logp, ref if with_ref else None, mask, cu, w, kind, beta, 0.0, 0.0, average)
    es = 3 * U * want[4] + U
    slope = beta + 2 * (want[5].abs() + 0.5 / beta) if kind == "squared" else torch.full_like(es, beta)
    _close(loss, want[0], slope * es * 2 + 16 * U * (1 + want[0].abs()) + 4 * U * slope * want[5].abs(), "loss")
    _close(reward, want[1], beta * es.repeat_interleave(2) * 2 + 2 * U * want[1].abs(), "reward")
    inside = torch.zeros(n, dtype=torch.bool, device="cuda")
    inside[int(cu[0]):int(cu[-1])] = True
    assert (dlogp[~inside] == 9).all() and (dlogp[inside & ~mask] == 0).all()
    pair = torch.bucketize(torch.arange(n, device="cuda"), cu[1:], right=True).clamp(max=2 * pairs - 1) // 2
    second = 2.0 if kind == "squared" else beta * beta
    tol = (second * es * 4)[pair] * w.double()[pair] + 24 * U * want[3].abs() + 24 * U * (slope * w.double())[pair]
    live = inside & mask
    if kind == "hinge":
        live &= ((want[5] * beta - 1).abs() > 4 * beta * es + 8 * U)[pair]
    _close(dlogp[live], want[3][live], tol[live], "dlogp")
