"""The AdamW step over a list of tensors where its states are NaN or infinite,
its eps is 0 or huge, its beta2 next to 1, or the sum of its gradients' squares
passes fp32's range.  The definition in fp32, one rounding per operation
(numpy), gives what must come out; a NaN may carry any bits."""
import math

import numpy as np
import pytest
import torch

import test_gpu_tensors as base
from test_gpu_tensors import BETA1, BETA2, BLOCK, EPS, F, LR, WD, _Case, _ctrl, _decode

pytestmark = pytest.mark.gpu

N = 6 * BLOCK + 77


def _definition(b, state, inv, eps=EPS, beta2=BETA2):
    """m', v' and the weights after the first step, in fp32."""
    c = lambda x: F(x)
    with np.errstate(all="ignore"):
        m = _decode(b["m"], b["ms"], True) if state == 8 else b["m"]
        v = _decode(b["v"], b["vs"], False) if state == 8 else b["v"]
        g = b["g"] * c(inv)
        m = c(BETA1) * m + c(1.0 - BETA1) * g
        v = c(beta2) * v + c(1.0 - beta2) * (g * g)
        u = (m / c(1.0 - BETA1)) / (np.sqrt(v / c(1.0 - beta2)) + c(eps))
        return b["th"] - c(LR) * (u + c(WD) * b["th"]), m, v


def _same(got, want, what):
    bad = (got.view(np.uint32) != want.view(np.uint32)) & ~(np.isnan(got) & np.isnan(want))
    assert not bad.any(), (what, int(bad.sum()), np.flatnonzero(bad)[:8], got[bad][:4], want[bad][:4])


def _step_and_check(zs, case, eps=EPS, beta2=BETA2, codes=False):
    before = case.host(0)
    zs.zero_tensors_adamw_async(case.list, zs.adam(LR, BETA1, beta2, eps, WD), _ctrl(zs, 1.0))
    th, m, v = _definition(before, case.state, 1.0, eps, beta2)
    got = case.host(0)
    _same(got["th"], th, "weights")
    if case.state == 32:
        _same(got["m"], m, "m")
        _same(got["v"], v, "v")
    elif codes:
        for name, x, signed in (("m", m, True), ("v", v, False)):
            code, scale = base._encode(x, signed)
            assert np.array_equal(got[name], code) and np.array_equal(got[name + "s"], scale), name
    return th


@pytest.mark.parametrize("lead", [0, 3])
@pytest.mark.parametrize("where", [0, 5, 300, N - 1])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("which", ["m", "v", "both"])
def test_nan_and_infinite_moments(zs, cuda_device, which, bad, where, lead):
    for quiet in (False, True):                # among usual values, and among zeros
        case = _Case(zs, [N], 32, torch.float32, None, 3, lead=lead)
        if quiet:
            for x in (case.grad, case.m, case.v):
                x[case.at[0]:case.at[0] + N] = 0
        if which != "v":
            case.m[case.at[0] + where] = bad
        if which != "m":
            case.v[case.at[0] + where] = bad
        th = _step_and_check(zs, case)
        assert np.isnan(th).sum() == (0 if (which, bad) == ("v", math.inf) or (which, bad) == ("m", math.inf) else 1)


@pytest.mark.parametrize("lead", [0, 5])
@pytest.mark.parametrize("scale", ["ms", "vs"])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_nan_and_infinite_scales_of_8_bit_states(zs, cuda_device, bad, scale, lead):
    case = _Case(zs, [N], 8, torch.bfloat16, None, 4, lead=lead)
    case.v[case.at[0] + 2 * BLOCK + 9] = 0     # 0 * inf
    case.m[case.at[0] + 2 * BLOCK + 9] = 0
    getattr(case, scale)[0][2] = bad
    th = _step_and_check(zs, case)
    assert np.isnan(th[2 * BLOCK + 9])


def test_a_huge_gradient_without_the_norm_pass(zs, cuda_device):
    """One gradient above 2^64: v' is infinite, and in the next step the states
    that are 0 decode to NaN, which the weights show."""
    case = _Case(zs, [N], 8, torch.float32, None, 5)
    case.grad[:N] = 0.0
    case.m[:N], case.v[:N] = 0, 0
    case.grad[BLOCK + 1] = 2.0 ** 65
    hp, ctrl = zs.adam(LR, BETA1, BETA2, EPS, WD), _ctrl(zs, 1.0)
    zs.zero_tensors_adamw_async(case.list, hp, ctrl)
    assert math.isinf(case.vs[0][1].item()) and case.master[:N].isfinite().all()
    case.grad[:N] = 0.01
    zs.zero_tensors_adamw_async(case.list, hp, ctrl)
    th = case.master[:N]
    assert th[BLOCK:2 * BLOCK].isnan().all() and th[:BLOCK].isfinite().all() and th[2 * BLOCK:].isfinite().all()


@pytest.mark.parametrize("state", [32, 8])
@pytest.mark.parametrize("lead", [0, 1, 7])
@pytest.mark.parametrize("eps", [0.0, 1e-60, 1e-30])
def test_eps_of_zero(zs, cuda_device, state, lead, eps):
    """Weights without gradient and states among others: 0 / 0 where eps is 0 in
    fp32, as one element at a time, whatever its neighbours are."""
    case = _Case(zs, [N], state, torch.float32, None, 6, lead=lead)
    at = case.at[0]
    for a, b in ((0, 3), (40, 45), (1024, 4096), (N - 5, N)):
        for x in (case.grad, case.m, case.v):
            x[at + a:at + b] = 0
    th = _step_and_check(zs, case, eps=eps, codes=True)
    assert np.isnan(th).any() == (F(eps) == 0)


@pytest.mark.parametrize("state", [32, 8])
@pytest.mark.parametrize("lead", [0, 7])
@pytest.mark.parametrize("eps", [1e10, 1e25, 1e38, 1e39, 1e300])
def test_eps_of_any_size(zs, cuda_device, state, lead, eps):
    """From 1e39 on it is infinite in fp32, and u is 0."""
    case = _Case(zs, [N], state, torch.float32, None, 6, lead=lead)
    for x in (case.grad, case.m, case.v):
        x[case.at[0] + 1024:case.at[0] + 4096] = 0
    assert np.isfinite(_step_and_check(zs, case, eps=eps, codes=True)).all()


@pytest.mark.parametrize("state", [32, 8])
@pytest.mark.parametrize("beta2", [1 - 2.0 ** -20, 1 - 2.0 ** -40, 1 - 2.0 ** -53])
def test_beta2_next_to_one(zs, cuda_device, state, beta2):
    """The bias correction of the first step is down to 2^-53."""
    case = _Case(zs, [N], state, torch.float32, None, 7)
    case.grad[:BLOCK] *= 1e4
    case.grad[BLOCK:2 * BLOCK] *= 1e-15
    if state == 32:
        case.v[:BLOCK] *= 1e15
        case.m[BLOCK:2 * BLOCK] *= 1e-20
        case.v[BLOCK:2 * BLOCK] = 1e12
    _step_and_check(zs, case, beta2=beta2, codes=True)


def test_squares_that_overflow_a_sum(zs, cuda_device):
    """Gradients just below the size that is refused one by one, 2^62: their sum
    passes the largest fp32.  Such a step may be skipped; it may not be taken
    unclipped."""
    n = 48_000_000
    grad = torch.full((n,), 2.0 ** 61 * 0.99, device="cuda")
    master, m, v = (torch.zeros(n, device="cuda") for _ in range(3))
    lst, ctrl, sq = zs.TensorList([zs.TensorView(grad, master, m, v)]), _ctrl(zs, 1.0), zs.new_sqnorm()
    zs.zero_tensors_sqnorm_async(lst, sq, zs.new_work(), ctrl)
    zs.zero_tensors_adamw_async(lst, zs.adam(LR), ctrl, max_norm=1.0, sqnorm_dev=sq)
    c = zs.read_ctrl(ctrl)
    if c["skipped"] == 0:
        # clipped to a norm of 1: m = (1 - beta1) / sqrt(n) everywhere
        assert abs(sq.item() / (n * grad[0].item() ** 2) - 1) < 1e-6
        assert abs(m[0].item() * math.sqrt(n) / 0.1 - 1) < 1e-5
    else:
        assert (m == 0).all() and c["step"] == 0
