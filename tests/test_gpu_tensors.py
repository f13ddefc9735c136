"""The AdamW step over a list of tensors, its norm pass and the values of 8-bit
states.  The update is compared bit for bit with the definition in fp32, one
rounding per operation (numpy), and with the flat shard step; and within the
roundings' sum with the definition in 64 bits."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BLOCK = 2048
F = np.float32
BETA1, BETA2, EPS, LR, WD = 0.9, 0.95, 1e-8, 3e-4, 0.1


def _map(bits):
    out = [0.0]
    for k in range(1, 1 << bits):
        f = k.bit_length() - 1
        out.append((0.1 + 0.9 * ((k - (1 << f) + 1) / (1 << f))) / 10.0 ** (bits - f - 1))
    return np.array(out, np.float32)


def _thresholds(table):
    mid = (table[1:].astype(np.float64) + table[:-1].astype(np.float64)) / 2
    t = mid.astype(np.float32)
    return np.where(t > mid, np.nextafter(t, F(0)), t)


M7, M8 = _map(7), _map(8)
T7, T8 = _thresholds(M7), _thresholds(M8)


def _decode(codes, scale, signed):
    table = np.concatenate([M7, -M7]) if signed else M8
    return table[codes] * np.repeat(scale, BLOCK)[:len(codes)]


def _encode(x, signed):
    n = len(x)
    blocks = -(-n // BLOCK)
    whole = np.zeros(blocks * BLOCK, np.float32)
    whole[:n] = x
    scale = np.abs(whole.reshape(-1, BLOCK)).max(1) if blocks else np.zeros(0, np.float32)
    q = whole.reshape(-1, BLOCK) / np.where(scale > 0, scale, F(1))[:, None]
    q = q.reshape(-1)[:n]
    code = np.searchsorted(T7 if signed else T8, np.abs(q), side="left").astype(np.uint8)
    if signed:
        code = np.where((q < 0) & (code > 0), code | 0x80, code).astype(np.uint8)
    return code, scale.astype(np.float32)


def _step32(g, th, m, v, t, inv, clip, lr=LR, wd=WD, dtype=np.float32):
    """One update, one rounding per operation in `dtype`."""
    c = lambda x: dtype(F(x))
    p1 = p2 = 1.0
    for _ in range(t):
        p1, p2 = p1 * BETA1, p2 * BETA2
    g = (g.astype(dtype) * c(inv)) * c(clip)
    m = c(BETA1) * m + c(1.0 - BETA1) * g
    v = c(BETA2) * v + c(1.0 - BETA2) * (g * g)
    u = (m / c(1.0 - p1)) / (np.sqrt(v / c(1.0 - p2)) + c(EPS))
    return th - c(lr) * (u + c(wd) * th), m, v


class _Case:
    """Tensors as parts of flat buffers, at any offsets."""

    def __init__(self, zs, numels, state, gtype, ptype, seed, lead=0, gap=0, scale=1.0, mults=None):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.zs, self.numels, self.state, self.ptype = zs, numels, state, ptype
        self.at = []
        pos = lead
        for n in numels:
            self.at.append(pos)
            pos += n + gap
        size = pos + 64
        r = lambda k=size: torch.randn(k, generator=g, device="cuda")
        self.grad = (r() * 0.02 * scale).to(gtype)
        self.master = r() * 0.05
        self.param = None if ptype is None else torch.zeros(size, dtype=ptype, device="cuda")
        self.mults = mults or [(1.0, 1.0)] * len(numels)
        blocks = [-(-n // BLOCK) for n in numels]
        if state == 8:
            self.m = torch.randint(0, 256, (size,), generator=g, device="cuda", dtype=torch.uint8)
            self.m[self.m == 128] = 0
            self.v = torch.randint(0, 256, (size,), generator=g, device="cuda", dtype=torch.uint8)
            self.ms = [torch.rand(b, generator=g, device="cuda") * 0.01 for b in blocks]
            self.vs = [torch.rand(b, generator=g, device="cuda") * 1e-4 for b in blocks]
        else:
            self.m, self.v = r() * 0.003, r().square() * 1e-5
            self.ms = self.vs = [None] * len(numels)
        part = lambda x, i: None if x is None else x[self.at[i]:self.at[i] + numels[i]]
        self.list = zs.TensorList([
            zs.TensorView(part(self.grad, i), part(self.master, i), part(self.m, i), part(self.v, i),
                          param=part(self.param, i), m_scale=self.ms[i], v_scale=self.vs[i], lr_mult=self.mults[i][0],
                          decay_mult=self.mults[i][1]) for i in range(len(numels))])
        self.part = part
        self.inside = torch.zeros(size, dtype=torch.bool, device="cuda")
        for a, n in zip(self.at, numels):
            self.inside[a:a + n] = True

    def flats(self):
        return [x for x in (self.grad, self.master, self.param, self.m, self.v) if x is not None]

    def host(self, i):
        n = lambda x: None if x is None else x.cpu().numpy().copy()
        out = dict(g=self.part(self.grad, i).float().cpu().numpy(), th=n(self.part(self.master, i)),
                   m=n(self.part(self.m, i)), v=n(self.part(self.v, i)), ms=n(self.ms[i]), vs=n(self.vs[i]),
                   p=None if self.param is None else self.part(self.param, i).cpu())
        return out


def _ctrl(zs, scale):
    c = zs.new_ctrl()
    zs.zero_ctrl_init(c, scale)
    return c


def _check_step(case, before, t, inv, clip):
    """Every tensor equals the fp32 definition bit for bit."""
    for i, b in enumerate(before):
        lr, wd = case.mults[i]
        m = _decode(b["m"], b["ms"], True) if case.state == 8 else b["m"]
        v = _decode(b["v"], b["vs"], False) if case.state == 8 else b["v"]
        th, m1, v1 = _step32(b["g"], b["th"], m, v, t, inv, clip, LR * lr, WD * wd)
        got = case.host(i)
        what = f"tensor {i} of {case.numels[i]} elements"
        assert np.array_equal(got["th"].view(np.uint32), th.view(np.uint32)), what
        if case.state == 8:
            for name, x, signed in (("m", m1, True), ("v", v1, False)):
                code, scale = _encode(x, signed)
                assert np.array_equal(got[name], code), (what, name)
                assert np.array_equal(got[name + "s"], scale), (what, name)
        else:
            assert np.array_equal(got["m"], m1) and np.array_equal(got["v"], v1), what
        if case.param is not None:
            assert torch.equal(got["p"], torch.from_numpy(th).to(case.ptype)), what


NUMELS = [1, 2, 7, 8, 9, 255, 256, 2047, 2048, 2049, 4096, 5000, 0, 12_345, 40_001]


@pytest.mark.parametrize("state", [32, 8])
@pytest.mark.parametrize("gtype,ptype", [(torch.bfloat16, torch.bfloat16), (torch.float16, torch.float16),
                                         (torch.float32, torch.bfloat16), (torch.float32, None)])
@pytest.mark.parametrize("lead,gap", [(0, 0), (3, 0), (1, 5), (0, 64)])
def test_step_matches_the_definition(zs, cuda_device, state, gtype, ptype, lead, gap):
    scale = 256.0 if gtype == torch.float16 else 1.0
    mults = [(1.0 + 0.25 * (i % 3), float(i % 2)) for i in range(len(NUMELS))]
    case = _Case(zs, NUMELS, state, gtype, ptype, 5 + state, lead, gap, scale, mults)
    ctrl, sq, work = _ctrl(zs, scale), zs.new_sqnorm(), zs.new_work()
    outside = [x[~case.inside].clone() for x in case.flats()]
    for t in (1, 2, 3):
        before = [case.host(i) for i in range(len(NUMELS))]
        zs.zero_tensors_sqnorm_async(case.list, sq, work, ctrl)
        norm = sum((b["g"].astype(np.float64) / scale).__pow__(2).sum() for b in before)
        # 8 squares to an fp32 sum (10 roundings), fp64 above that
        assert abs(sq.item() - norm) <= 12 * U * norm
        zs.zero_tensors_adamw_async(case.list, zs.adam(LR, BETA1, BETA2, EPS, WD), ctrl, max_norm=0.5, sqnorm_dev=sq)
        clip = F(min(1.0, 0.5 / (math.sqrt(sq.item()) + 1e-6)))
        _check_step(case, before, t, 1.0 / scale, clip)
        c = zs.read_ctrl(ctrl)
        assert c["step"] == t and c["skipped"] == 0 and c["arrivals"] == 0
    for a, x in zip(outside, case.flats()):
        assert torch.equal(a, x[~case.inside]), "written outside the tensors"


def test_step_within_the_roundings_of_64_bits(zs, cuda_device):
    """m: 3 roundings of its terms and 2 of g; v: 4 and 4; the update u: m's and
    half of v's relative errors, and 6 roundings of its own, times lr."""
    case = _Case(zs, [30_000], 32, torch.bfloat16, None, 1)
    b, ctrl = case.host(0), _ctrl(zs, 1.0)
    zs.zero_tensors_adamw_async(case.list, zs.adam(LR, BETA1, BETA2, EPS, WD), ctrl)
    d = lambda x: x.astype(np.float64)
    g = d(b["g"])
    m, v = BETA1 * d(b["m"]) + (1 - BETA1) * g, BETA2 * d(b["v"]) + (1 - BETA2) * g * g
    mh, den = m / (1 - BETA1), np.sqrt(v / (1 - BETA2)) + EPS
    th = d(b["th"]) - LR * (mh / den + WD * d(b["th"]))
    got = case.host(0)
    em = 6 * U * (np.abs(BETA1 * d(b["m"])) + (1 - BETA1) * np.abs(g))
    assert (np.abs(got["m"] - m) <= em).all()
    assert (np.abs(got["v"] - v) <= 9 * U * v).all()
    eu = em / (1 - BETA1) / den + np.abs(mh / den) * 12 * U
    assert (np.abs(got["th"] - th) <= LR * (eu + 4 * U * (np.abs(mh / den) + 1)) + 2 * U * (np.abs(th) + LR * np.abs(mh / den))).all()


@pytest.mark.parametrize("state", [32, 8])
def test_matches_the_shard_step_bit_for_bit(zs, cuda_device, state):
    """One fp16 contribution, no clipping: the list's step and the flat shard
    step are the same arithmetic."""
    n, scale = 100_003, 1024.0
    case = _Case(zs, [n], state, torch.float16, torch.float16, 9, scale=scale)
    hp, ctrl, other = zs.adam(LR, BETA1, BETA2, EPS, WD), _ctrl(zs, scale), _ctrl(zs, scale)
    copy = lambda x: [x[:n].clone(), torch.empty_like(x[:n])]
    if state == 8:
        pair = lambda x: [x.clone(), torch.empty_like(x)]
        shard = zs.Adam8View([case.grad[:n].contiguous()], copy(case.master), copy(case.m), copy(case.v),
                             pair(case.ms[0]), pair(case.vs[0]), torch.zeros(n, dtype=torch.float16, device="cuda"), n)
        step = lambda: zs.zero_shard_step_adam8_async([shard], 1, hp, other)
    else:
        shard = zs.ShardView([case.grad[:n].contiguous()], copy(case.master), copy(case.m), copy(case.v),
                             torch.zeros(n, dtype=torch.float16, device="cuda"), n)
        step = lambda: zs.zero_shard_step_async([shard], 1, hp, other)
    for t in range(1, 5):
        zs.zero_tensors_adamw_async(case.list, hp, ctrl)
        step()
        cur = zs.read_ctrl(other)["cur"]
        assert torch.equal(case.master[:n], shard.master[cur]) and torch.equal(case.param[:n], shard.params)
        if state == 8:
            assert torch.equal(case.m[:n], shard.m_codes[cur]) and torch.equal(case.v[:n], shard.v_codes[cur])
            assert torch.equal(case.ms[0], shard.m_scale[cur]) and torch.equal(case.vs[0], shard.v_scale[cur])
        else:
            assert torch.equal(case.m[:n], shard.m[cur]) and torch.equal(case.v[:n], shard.v[cur])


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan, 2.0 ** 63])
@pytest.mark.parametrize("state", [32, 8])
def test_non_finite_gradient_skips_the_step(zs, cuda_device, bad, state):
    case = _Case(zs, [5, 3000, 70], state, torch.float32, torch.bfloat16, 2)
    ctrl, sq, work, hp = _ctrl(zs, 8.0), zs.new_sqnorm(), zs.new_work(), zs.adam(LR)
    place = case.at[1] + 2999
    good = case.grad[place].item()
    case.grad[place] = bad * 8.0
    before = [x.clone() for x in case.flats()[1:]] + [x.clone() for x in case.ms + case.vs if x is not None]
    zs.zero_tensors_sqnorm_async(case.list, sq, work, ctrl)
    zs.zero_tensors_adamw_async(case.list, hp, ctrl, max_norm=1.0, sqnorm_dev=sq)
    after = case.flats()[1:] + [x for x in case.ms + case.vs if x is not None]
    for a, b in zip(before, after):
        assert torch.equal(a.nan_to_num(), b.nan_to_num())
    c = zs.read_ctrl(ctrl)
    assert (c["skipped"], c["step"], c["loss_scale"], c["overflow"], c["last_overflow"]) == (1, 0, 4.0, 0, 1)
    case.grad[place] = good
    zs.zero_tensors_sqnorm_async(case.list, sq, work, ctrl)
    zs.zero_tensors_adamw_async(case.list, hp, ctrl, max_norm=1.0, sqnorm_dev=sq)
    c = zs.read_ctrl(ctrl)
    assert (c["skipped"], c["step"], c["last_overflow"]) == (1, 1, 0)
    assert not torch.equal(before[0], case.master)


@pytest.mark.parametrize("state", [32, 8])
def test_more_tensors_than_one_launch_takes(zs, cuda_device, state):
    r = np.random.Generator(np.random.PCG64(3))
    numels = [int(x) for x in np.exp(r.random(2500) * math.log(3000))]
    case = _Case(zs, numels, state, torch.bfloat16, torch.bfloat16, 4)
    ctrl, sq, work = _ctrl(zs, 1.0), zs.new_sqnorm(), zs.new_work()
    before = [case.host(i) for i in range(len(numels))]
    zs.zero_tensors_sqnorm_async(case.list, sq, work, ctrl)
    first = sq.item()
    zs.zero_tensors_sqnorm_async(case.list, sq, work, ctrl)
    assert sq.item() == first, "the order of the sum is fixed"
    norm = sum((b["g"].astype(np.float64) ** 2).sum() for b in before)
    assert abs(first - norm) <= 12 * U * norm
    zs.zero_tensors_adamw_async(case.list, zs.adam(LR, BETA1, BETA2, EPS, WD), ctrl)
    _check_step(case, before, 1, 1.0, 1.0)
    assert zs.read_ctrl(ctrl)["step"] == 1


def test_both_kinds_of_state_and_empty_tensors_in_one_step(zs, cuda_device):
    a = _Case(zs, [0, 3000, 17], 8, torch.bfloat16, None, 1)
    b = _Case(zs, [2500, 0], 32, torch.float32, torch.float16, 2)
    both = zs.TensorList([v for pair in zip(a.list.views[:2], b.list.views) for v in pair] + a.list.views[2:])
    ctrl = _ctrl(zs, 1.0)
    before = [[c.host(i) for i in range(len(c.numels))] for c in (a, b)]
    zs.zero_tensors_adamw_async(both, zs.adam(LR, BETA1, BETA2, EPS, WD), ctrl)
    for c, old in zip((a, b), before):
        _check_step(c, old, 1, 1.0, 1.0)
    assert zs.read_ctrl(ctrl)["step"] == 1
    empty = zs.TensorList([a.list.views[0], b.list.views[1]])
    sq = zs.new_sqnorm() + 5
    zs.zero_tensors_sqnorm_async(empty, sq, zs.new_work(), ctrl)
    zs.zero_tensors_adamw_async(empty, zs.adam(LR), ctrl)
    c = zs.read_ctrl(ctrl)
    assert sq.item() == 0.0 and c["step"] == 2 and c["arrivals"] == 0


@pytest.mark.parametrize("peel", range(8))
def test_eight_bit_blocks_at_every_alignment(zs, cuda_device, peel):
    """Blocks count from the tensor's start, vectors from the buffers'."""
    case = _Case(zs, [9000 + peel], 8, torch.bfloat16, torch.bfloat16, peel, lead=peel)
    ctrl = _ctrl(zs, 1.0)
    for t in (1, 2):
        before = [case.host(0)]
        zs.zero_tensors_adamw_async(case.list, zs.adam(LR, BETA1, BETA2, EPS, WD), ctrl)
        _check_step(case, before, t, 1.0, 1.0)


@pytest.mark.parametrize("state", [32, 8])
def test_buffers_that_share_no_boundary(zs, cuda_device, state):
    n = 7001
    case = _Case(zs, [n], state, torch.float16, torch.bfloat16, 6)
    shift = lambda x, k: torch.cat([x[:k], x[:n]])[k:]
    g, m, v = shift(case.grad, 3), shift(case.m, 1), shift(case.v, 5)
    old = case.list.views[0]
    moved = zs.TensorView(g, old.master, m, v, param=old.param, m_scale=old.m_scale, v_scale=old.v_scale)
    before = [case.host(0)]
    zs.zero_tensors_adamw_async(zs.TensorList([moved]), zs.adam(LR, BETA1, BETA2, EPS, WD), _ctrl(zs, 1.0))
    case.m[:n], case.v[:n] = m, v
    _check_step(case, before, 1, 1.0, 1.0)


def test_eight_bit_extreme_scales(zs, cuda_device):
    """Blocks whose largest state is zero, tiny (a subnormal quotient's divisor)
    or huge take the same codes as the division."""
    n = 6 * BLOCK
    case = _Case(zs, [n], 8, torch.float32, None, 8)
    case.grad[:BLOCK] = 0.0
    case.m[:BLOCK], case.v[:BLOCK] = 0, 0
    for i, s in enumerate((1e-18, 1e-30, 1e12, 1e-3, 1e-8), 1):
        case.grad[i * BLOCK:(i + 1) * BLOCK] *= s
        case.ms[0][i] = s * 0.01
        case.vs[0][i] = s * s * 1e-3
    before = [case.host(0)]
    zs.zero_tensors_adamw_async(case.list, zs.adam(LR, BETA1, BETA2, EPS, WD), _ctrl(zs, 1.0))
    with np.errstate(all="ignore"):
        _check_step(case, before, 1, 1.0, 1.0)


@pytest.mark.parametrize("state", [32, 8])
def test_weights_without_gradients_and_states(zs, cuda_device, state):
    """Rows of zeros (m = v = g = 0) next to others: u = 0 there, and the weights
    only decay."""
    n = 20_000
    case = _Case(zs, [n], state, torch.bfloat16, torch.bfloat16, 12)
    zero = torch.arange(n, device="cuda") % 1000 < 700
    zero[5000:5003] = True
    for x in (case.grad, case.m, case.v):
        x[:n][zero] = 0
    before = [case.host(0)]
    zs.zero_tensors_adamw_async(case.list, zs.adam(LR, BETA1, BETA2, EPS, WD), _ctrl(zs, 1.0))
    _check_step(case, before, 1, 1.0, 1.0)
    # v' of 0 with an m' that is not
    case = _Case(zs, [n], state, torch.float32, None, 13)
    case.grad[:n] = 1e-30
    case.v[:n] = 0
    before = [case.host(0)]
    with np.errstate(all="ignore"):
        zs.zero_tensors_adamw_async(case.list, zs.adam(LR, BETA1, BETA2, EPS, WD), _ctrl(zs, 1.0))
        _check_step(case, before, 1, 1.0, 1.0)


@pytest.mark.parametrize("n,shift", [(1, 0), (7, 0), (2048, 0), (5001, 0), (5001, 1), (1_000_003, 0)])
@pytest.mark.parametrize("signed", [True, False])
def test_values_of_8_bit_states(zs, cuda_device, n, shift, signed):
    g = torch.Generator(device="cuda")
    g.manual_seed(n)
    codes = torch.randint(0, 256, (n + shift,), generator=g, device="cuda", dtype=torch.uint8)[shift:]
    scales = torch.rand(-(-n // BLOCK), generator=g, device="cuda")
    out = torch.full((n + 8,), 3.0, device="cuda")
    zs.zero_adam8_dequantize(codes, scales, n, signed, out)
    want = _decode(codes.cpu().numpy(), scales.cpu().numpy(), signed)
    assert np.array_equal(out[:n].cpu().numpy(), want) and (out[n:] == 3).all()


def test_tensor_offsets_past_32_bits(zs, cuda_device):
    """One tensor of 2^31 + 5000 elements with 8-bit states: its last block."""
    n = (1 << 31) + 5000
    grad = torch.full((n,), 0.01, dtype=torch.bfloat16, device="cuda")
    master = torch.full((n,), 0.5, device="cuda")
    m, v = (torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in range(2))
    ms, vs = (torch.zeros(-(-n // BLOCK), device="cuda") for _ in range(2))
    grad[-3:] = torch.tensor([0.02, -0.03, 0.0], device="cuda").to(torch.bfloat16)
    lst, ctrl, sq = zs.TensorList([zs.TensorView(grad, master, m, v, m_scale=ms, v_scale=vs)]), _ctrl(zs, 1.0), zs.new_sqnorm()
    zs.zero_tensors_sqnorm_async(lst, sq, zs.new_work(), ctrl)
    zs.zero_tensors_adamw_async(lst, zs.adam(LR, BETA1, BETA2, EPS, 0.0), ctrl)
    one = grad[0].item()
    tail = grad[-3:].double().square().sum().item()
    assert abs(sq.item() - ((n - 3) * one * one + tail)) <= 12 * U * n * one * one
    first = (n - 1) // BLOCK * BLOCK
    g = grad[first:].float().cpu().numpy()
    zero = np.zeros_like(g)
    th, m1, v1 = _step32(g, np.full_like(g, 0.5), zero, zero, 1, 1.0, 1.0, LR, 0.0)
    assert np.array_equal(master[first:].cpu().numpy(), th)
    code, scale = _encode(m1, True)
    assert np.array_equal(m[first:].cpu().numpy(), code) and ms[-1].item() == scale[0]
    code, scale = _encode(v1, False)
    assert np.array_equal(v[first:].cpu().numpy(), code) and vs[-1].item() == scale[0]
    assert (master[: 1 << 20] == master[0]).all() and master[1 << 31].item() == master[0].item()
