"""The policy loss where a log-probability is infinite: a token that the reference
model, or the model itself, gives no chance.  Without a coefficient the KL term is
no part of the loss or of its gradient, whatever its value is."""
import math

import pytest
import torch

from test_gpu_losses import HALF_UNIT, TINY, U, _close, _err, _policy_inputs

pytestmark = pytest.mark.gpu

INF = math.inf
ROWS, V = 6, 1200


def _run(zs, x, y, old, adv, hp, ref):
    f = lambda *n: torch.full(n, 9.0, device="cuda")
    logp, loss, totals, out = f(len(y)), f(len(y)), f(5), torch.full_like(x, 9.0)
    zs.zero_policy_loss_async(x, y, old, adv, None, zs.policy(**hp), totals, zs.new_work(), ref_logp=ref, logp=logp,
                              token_loss=loss, dlogits=out)
    return logp, loss, totals, out


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_kl_without_a_coefficient(zs, cuda_device, dtype):
    x, y, old, ref, adv, _ = _policy_inputs(ROWS, V, dtype, 3)
    x[1, y[1]] = -INF                   # the model itself: ratio 0
    ref[2], ref[3] = -INF, INF
    want = _run(zs, x, y, old, adv, {}, None)
    got = _run(zs, x, y, old, adv, {}, ref)
    assert want[1].isfinite().all() and want[3].isfinite().all()
    for i in (0, 1, 3):
        assert torch.equal(got[i], want[i])
    for i in (0, 1, 3, 4):
        assert got[2][i].item() == want[2][i].item()
    # the KL itself is infinite: e^gap - gap - 1 with gap of +inf or -inf
    assert got[2][2].item() == INF


@pytest.mark.parametrize("kl", [0.1, 2.0])
def test_kl_with_a_coefficient(zs, cuda_device, kl):
    """A reference of -inf: the loss is +inf and its gradient finite, that of
    pg + kl (-gap - 1)."""
    x, y, old, ref, adv, _ = _policy_inputs(ROWS, V, torch.float32, 4)
    ref[:] = -INF
    logp, loss, totals, out = _run(zs, x, y, old, adv, {"kl_coef": kl}, ref)
    assert (loss == INF).all() and totals[0].item() == INF and totals[2].item() == INF
    plain = _run(zs, x, y, old, adv, {}, None)[3].double()
    p = torch.softmax(x.double(), 1)
    hot = torch.zeros_like(p).scatter_(1, y[:, None], 1.0)
    more = kl / ROWS * (hot - p)
    e = _err(V)
    tol = (2 * e + 320 * U) * 4 * ((plain.abs() + kl / ROWS * (p + hot))) + HALF_UNIT[torch.float32] * 4 * (plain + more).abs() + TINY[torch.float32]
    _close(out, plain + more, tol, "dlogits")


@pytest.mark.parametrize("dual", [0.0, 3.0])
def test_a_ratio_past_fp32(zs, cuda_device, dual):
    """logp - old_logp of 100: exp passes fp32.  With A = 0 the loss and its
    gradient are 0; with A > 0 the clipped bound holds; with A < 0 the loss is
    past fp32 too, or capped."""
    x, y, _, _, _, _ = _policy_inputs(ROWS, V, torch.float32, 5)
    logp64 = torch.log_softmax(x.double(), 1).gather(1, y[:, None])[:, 0]
    old = (logp64 - 100.0).float()
    adv = torch.tensor([0.0, 1.0, -1.0, -0.0, 0.5, 0.0], device="cuda")
    old[5] = -INF
    logp, loss, totals, out = _run(zs, x, y, old, adv, {"dual_clip": dual}, None)
    want = [0.0, -1.2, 3.0 if dual else INF, 0.0, -0.6, 0.0]
    for i, w in enumerate(want):
        assert loss[i].item() == w or abs(loss[i].item() - w) <= 4 * U * abs(w), i
    still = [0, 1, 3, 4, 5] + ([2] if dual else [])
    assert (out[still] == 0).all()
