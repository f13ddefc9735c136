"""The preference loss where a sequence's score is infinite: a token that the
model gives no chance (log-probability -inf) or the reference does not.  The
definition has a value there: with h = +inf the sigmoid loss is 0 without and
+inf with label smoothing, the hinge loss 0, the squared one +inf; and the
gradients are those of the formula at z = +-inf."""
import math

import pytest
import torch

from test_gpu_losses import U, _close

pytestmark = pytest.mark.gpu

INF = math.inf
BETA, W = 0.25, 0.5


def _scalars(kind, ls, h):
    """loss and d loss / d h."""
    z = BETA * h
    if kind == "sigmoid":
        soft = lambda t: max(t, 0.0) + math.log1p(math.exp(-abs(t)))
        loss = (1 - ls) * soft(-z) + (ls * soft(z) if ls else 0.0)
        sig = lambda t: 0.0 if t == -INF else 1.0 if t == INF else 1 / (1 + math.exp(-t))
        return loss, BETA * (ls * sig(z) - (1 - ls) * sig(-z))
    if kind == "hinge":
        return max(0.0, 1.0 - z), -BETA if z < 1 else 0.0
    return (h - 0.5 / BETA) ** 2, 2 * (h - 0.5 / BETA)


@pytest.mark.parametrize("kind,ls", [("sigmoid", 0.0), ("sigmoid", 0.2), ("hinge", 0.0), ("squared", 0.0)])
@pytest.mark.parametrize("average", [False, True])
@pytest.mark.parametrize("length", [1, 3, 10, 4000, 100_000])
@pytest.mark.parametrize("offset", [0, 1])
def test_infinite_scores(zs, cuda_device, kind, ls, average, length, offset):
    # pairs: an impossible token chosen, rejected, impossible to the reference
    # (chosen, rejected), in both (no value), and an ordinary pair
    pairs = 6
    n = 2 * pairs * length
    g = torch.Generator(device="cuda")
    g.manual_seed(length)
    logp = torch.full((n + offset,), -1.0, device="cuda")[offset:]
    ref = torch.full((n,), -1.0, device="cuda")
    at = [int(torch.randint(0, length, (1,), generator=g, device="cuda")) for _ in range(2 * pairs)]
    place = lambda s: s * length + at[s]
    logp[place(0)] = -INF
    logp[place(3)] = -INF
    ref[place(4)] = -INF
    ref[place(7)] = -INF
    logp[place(8)] = logp[place(9)] = -INF
    cu = torch.arange(0, n + 1, length, device="cuda")
    w = torch.full((pairs,), W, device="cuda")
    f = lambda k: torch.full((k,), 9.0, device="cuda")
    loss, reward, totals, dlogp, work = f(pairs), f(2 * pairs), f(3), f(n), zs.new_work()
    hp = zs.preference(BETA, kind, ls, 0.0, average)
    run = lambda wt: zs.zero_preference_loss_async(logp, cu, hp, loss, reward, totals, work, ref_logp=ref, weights=wt, dlogp=dlogp)
    run(w)
    share = 1.0 / length if average else 1.0
    for i, s in enumerate([(-INF, 0.0), (0.0, -INF), (INF, 0.0), (0.0, INF), (-INF, -INF), (0.0, 0.0)]):
        assert reward[2 * i:2 * i + 2].tolist() == [BETA * t for t in s], i
        if i == 4:
            assert math.isnan(loss[i].item())
            continue
        want, dh = _scalars(kind, ls, s[0] - s[1])
        _close(loss[i:i + 1], torch.tensor([want], dtype=torch.float64, device="cuda"), 16 * U * (1 + abs(want) if want < INF else 1), f"loss of pair {i}")
        for k, sign in ((0, 1.0), (1, -1.0)):
            part = dlogp[(2 * i + k) * length:(2 * i + k + 1) * length].double()
            d = torch.full_like(part, sign * dh * share * W)
            _close(part, d, 16 * U * d.abs().nan_to_num(0, 0, 0), f"dlogp of pair {i}")
    # only the pair without a value spoils the totals; without it they are the definition's
    w[4] = 0.0
    run(w)
    each = [_scalars(kind, ls, h)[0] for h in (-INF, INF, INF, -INF, 0.0)]
    want = W * sum(each)
    assert totals[0].item() == want or abs(totals[0].item() - want) <= 64 * U * (1 + want)
    assert totals[1].item() == 2 * W


def test_infinities_of_both_signs_have_no_score(zs, cuda_device):
    x = torch.tensor([-INF, INF, -1.0, -1.0], device="cuda")
    cu = torch.tensor([0, 2, 4], device="cuda")
    f = lambda k: torch.full((k,), 9.0, device="cuda")
    loss, reward, totals = f(1), f(2), f(3)
    zs.zero_preference_loss_async(x, cu, zs.preference(0.5), loss, reward, totals, zs.new_work())
    assert reward[0].isnan() and reward[1].item() == -1.0 and loss[0].isnan()
