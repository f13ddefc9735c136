"""Workloads of the fine-tuning operators: token log-probabilities, the clipped
policy loss, the preference loss and the AdamW step over a list of tensors.

``listed()`` and ``draw()`` name the cases, ``prepare()`` makes a case's inputs
on the GPU, ``run()`` makes one pass: with ``own`` the calls of the framework,
otherwise the same operator in elementary 32-bit torch operations.
``exact()`` is the definition in 64 bits.
"""
import math
import random

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
BLOCK = 2048                       # elements per scale of the 8-bit states
BETA1, BETA2, EPS = 0.9, 0.95, 1e-8
LR, DECAY, MAX_NORM = 3e-4, 0.1, 1.0
SCALE = 1024.0                     # loss scale carried by fp16 gradients
MOST_LOGITS = 1 << 30
MOST_TOKENS = 1 << 23
MOST_NUMEL = 400_000_000


# ------------------------------------------------------------------- cases ---

def listed():
    return [
        # scoring the four sequences' current tokens of a small sampler, fp32 logits: latency
        {"name": "logp small", "op": "logp", "rows": 4, "vocab": 32000, "pad": 0, "type": "f32",
         "ignored": 0.0, "banned": 0.0, "entropy": True, "temperature": 0.7},
        # scoring a packed batch; an odd vocabulary, rows not aligned to vector accesses
        {"name": "logp batch", "op": "logp", "rows": 8192, "vocab": 50257, "pad": 0, "type": "bf16",
         "ignored": 0.25, "banned": 0.0, "entropy": False, "temperature": 1.0},
        # backward of scoring in a preference step, with an entropy gradient
        {"name": "logp gradient", "op": "logp_grad", "rows": 3000, "vocab": 32000, "pad": 0, "type": "f16",
         "ignored": 0.4, "banned": 0.0, "entropy": True, "temperature": 1.0},
        # one short answer: latency again, forward and backward
        {"name": "policy small", "op": "policy", "rows": 24, "vocab": 50257, "pad": 47, "type": "f16",
         "ignored": 0.1, "banned": 0.01, "entropy": True, "temperature": 1.0},
        # a usual micro-batch, prompts masked out
        {"name": "policy batch", "op": "policy", "rows": 4096, "vocab": 32000, "pad": 0, "type": "bf16",
         "ignored": 0.3, "banned": 0.0, "entropy": False, "temperature": 1.0},
        # a large micro-batch of a large vocabulary
        {"name": "policy large", "op": "policy", "rows": 8192, "vocab": 131072, "pad": 0, "type": "bf16",
         "ignored": 0.1, "banned": 0.0, "entropy": True, "temperature": 0.9},
        # one micro-batch of four pairs
        {"name": "preference small", "op": "preference", "pairs": 4, "mean": 200, "type": "f32",
         "ignored": 0.3, "kind": "sigmoid", "average": False, "ref": True},
        # a whole epoch's scores at once: long and short answers mixed
        {"name": "preference large", "op": "preference", "pairs": 4096, "mean": 1000, "type": "f32",
         "ignored": 0.3, "kind": "sigmoid", "average": False, "ref": True},
        # adapters and norms: few and small tensors, latency
        {"name": "adamw small", "op": "adamw", "sizes": "loguniform", "tensors": 30, "max_numel": 1 << 14,
         "sizes_seed": 3, "state": 32, "type": "bf16", "copy": "bf16", "packed": False, "clip": True},
        # many tensors of all sizes, packed end to end in flat buffers (odd offsets)
        {"name": "adamw ragged", "op": "adamw", "sizes": "loguniform", "tensors": 1200, "max_numel": 1 << 20,
         "sizes_seed": 7, "state": 32, "type": "bf16", "copy": "bf16", "packed": True, "clip": True},
        # 8-bit states of a small model
        {"name": "adamw 8-bit small", "op": "adamw", "sizes": "loguniform", "tensors": 100, "max_numel": 1 << 19,
         "sizes_seed": 11, "state": 8, "type": "bf16", "copy": "bf16", "packed": False, "clip": False},
        # 8-bit states of embeddings, two layers (4096 wide, 11008 in the middle) and a head
        {"name": "adamw 8-bit large", "op": "adamw", "sizes": "layers", "tensors": 21, "max_numel": 0,
         "sizes_seed": 0, "state": 8, "type": "f16", "copy": "f16", "packed": False, "clip": False},
    ]


def _log_between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logp", "logp_grad", "policy", "policy", "preference", "adamw", "adamw"])
    if op == "preference":
        pairs = _log_between(rng, 1, 4096)
        return {"op": op, "pairs": pairs, "mean": _log_between(rng, 4, min(30000, MOST_TOKENS // (2 * pairs))),
                "type": "f32", "ignored": rng.choice([0.0, 0.3, 0.9]),
                "kind": rng.choice(["sigmoid", "hinge", "squared"]), "average": rng.random() < 0.4,
                "ref": rng.random() < 0.7}
    if op == "adamw":
        state = rng.choice([8, 32])
        return {"op": op, "sizes": "loguniform", "tensors": _log_between(rng, 1, 1200),
                "max_numel": _log_between(rng, 100, 1 << 20), "sizes_seed": rng.randrange(1 << 20), "state": state,
                "type": rng.choice(["bf16", "f16", "f32"]), "copy": rng.choice(["bf16", "f16", "none"]),
                "packed": state == 32 and rng.random() < 0.5, "clip": state == 32}
    vocab = _log_between(rng, 500, 200_000)
    return {"op": op, "rows": _log_between(rng, 1, min(12_000, MOST_LOGITS // (2 * vocab))), "vocab": vocab,
            "pad": rng.choice([0, 0, rng.randrange(1, 130)]), "type": rng.choice(["bf16", "f16", "f32"]),
            "ignored": rng.choice([0.0, 0.3, 0.8]), "banned": rng.choice([0.0, 0.0, 0.2]),
            "entropy": rng.random() < 0.5, "temperature": rng.choice([1.0, 0.7, 1.3])}


def _numels(case):
    if case["sizes"] == "layers":
        d, ffn, vocab = 4096, 11008, 32000
        out = [vocab * d]
        for _ in range(2):
            out += [d * d] * 4 + [ffn * d] * 3 + [d] * 2
        return out + [d, vocab * d]
    r = random.Random(case["sizes_seed"])
    out, left = [], MOST_NUMEL
    for _ in range(case["tensors"]):
        n = min(left, max(1, int(math.exp(r.uniform(0.0, math.log(case["max_numel"]))))))
        out.append(max(n, 1))
        left = max(0, left - n)
    return out


def _offsets(case, numels):
    """First element of each tensor in the flat buffers, and their length: end to
    end, or each on a boundary (a scale block's, for 8-bit states)."""
    step = 1 if case["packed"] else BLOCK if case["state"] == 8 else 64
    at, out = 0, []
    for n in numels:
        out.append(at)
        at += -(-n // step) * step
    return out, at


# ------------------------------------------------------------------ inputs ---

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda")


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _logits(case, g):
    """Logits of spread 2.5 in which each row's label stands out by 0 to 9; a
    share of the labels ignored; a share of the vocabulary banned (-inf)."""
    t, v = case["rows"], case["vocab"]
    full = torch.empty(t, v + case["pad"], dtype=TYPES[case["type"]], device="cuda")
    labels = torch.randint(0, v, (t,), generator=g, device="cuda")
    boost = _rand(g, t) * 9.0
    banned = _rand(g, v) < case["banned"]
    true_logp = torch.empty(t, device="cuda")
    step = max(1, (1 << 26) // v)
    for a in range(0, t, step):
        b = min(t, a + step)
        x = _randn(g, b - a, v + case["pad"]) * 2.5
        row = torch.arange(b - a, device="cuda")
        keep = x[row, labels[a:b]] + boost[a:b]
        x[:, :v].masked_fill_(banned, -math.inf)
        x[row, labels[a:b]] = keep
        full[a:b] = x
        z = full[a:b, :v].float() / case["temperature"]
        true_logp[a:b] = z[row, labels[a:b]] - torch.logsumexp(z, 1)
    skip = _rand(g, t) < case["ignored"]
    return full[:, :v], labels, skip, true_logp


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case, "it": 1.0 / case.get("temperature", 1.0)}
    if case["op"] == "preference":
        p = case["pairs"]
        # lengths of an exponential spread (some of them 0 or 1) that fill the list of tokens
        s["n"] = n = 2 * p * case["mean"]
        ends = _rand(g, 2 * p).clamp(min=1e-6).log().neg().double().cumsum(0)
        s["cu"] = torch.zeros(2 * p + 1, dtype=torch.int64, device="cuda")
        s["cu"][1:] = (ends * (n / ends[-1])).round().long()
        s["cu"][-1] = n
        lens = s["cu"][1:] - s["cu"][:-1]
        s["longest"] = int(lens.max())
        s["logp"] = _rand(g, n).clamp(min=1e-6).log() * 1.5
        s["ref"] = s["logp"] + _randn(g, n) * 0.05 if case["ref"] else None
        s["mask"] = _rand(g, n) >= case["ignored"]
        # without a reference or an average the sums are long: a smaller beta keeps them in the loss's range
        s["beta"] = 0.1 if case["ref"] else 2.0 if case["average"] else 0.002
        s["margin"] = 0.0 if case["ref"] else 0.3
    elif case["op"] == "adamw":
        s["numels"] = numels = _numels(case)
        s["offsets"], s["n"] = _offsets(case, numels)
        n = s["n"]
        s["loss_scale"] = SCALE if case["type"] == "f16" else 1.0
        inside = torch.zeros(n, dtype=torch.bool, device="cuda")
        for at, k in zip(s["offsets"], numels):
            inside[at:at + k] = True
        s["grad"] = (_randn(g, n) * (2e-3 * s["loss_scale"])).to(TYPES[case["type"]]) * inside
        s["master"] = _randn(g, n) * 0.02 * inside
        s["copy"] = None if case["copy"] == "none" else s["master"].to(TYPES[case["copy"]])
        s["spans"] = torch.tensor([b - a for a, b in zip(s["offsets"], s["offsets"][1:] + [n])], device="cuda")
        # weights decay, vectors (here: small tensors) do not
        s["decay"] = [1.0 if k > 5000 else 0.0 for k in numels]
        s["beta_pow"] = [1.0, 1.0]
        if case["state"] == 8:
            blocks = n // BLOCK
            s["m"] = torch.zeros(n, dtype=torch.uint8, device="cuda")
            s["v"] = torch.zeros(n, dtype=torch.uint8, device="cuda")
            s["m_scale"] = torch.zeros(blocks, device="cuda")
            s["v_scale"] = torch.zeros(blocks, device="cuda")
            # states as they are after some steps: codes over the whole map
            s["m"][:] = torch.randint(0, 256, (n,), generator=g, device="cuda", dtype=torch.uint8) * inside
            s["m"][s["m"] == 128] = 0
            s["v"][:] = torch.randint(60, 256, (n,), generator=g, device="cuda", dtype=torch.uint8) * inside
            s["m_scale"][:] = 2e-3 + 1e-3 * _rand(g, blocks)
            s["v_scale"][:] = 1e-5 + 1e-5 * _rand(g, blocks)
        else:
            s["m"] = _randn(g, n) * 5e-4 * inside
            s["v"] = _randn(g, n).square() * 4e-6 * inside
        del inside
    else:
        s["x"], s["labels"], skip, logp = _logits(case, g)
        t = case["rows"]
        s["logp"] = logp
        if case["op"] == "policy":
            s["weights"] = (~skip).float() / max(1, t)
            noise = _randn(g, t) * 0.2
            # off the edges of the clipped range, where 32-bit forms may fall on either side
            for edge in (math.log(0.8), math.log(1.28), math.log(3.0)):
                noise = torch.where((noise - edge).abs() < 2e-3, noise + 5e-3, noise)
            s["old"] = logp - noise
            s["ref"] = logp + _randn(g, t) * 0.3
            s["adv"] = _randn(g, t)
            s["coef"] = {"clip_low": 0.2, "clip_high": 0.28, "dual_clip": 3.0, "kl_coef": 0.05,
                         "entropy_coef": 0.01 if case["entropy"] else 0.0}
            s["loss_scale"] = SCALE if case["type"] == "f16" else 1.0
        else:
            s["labels"] = torch.where(skip, torch.full_like(s["labels"], -100), s["labels"])
        if case["op"] == "logp_grad":
            s["dlogp"] = _randn(g, t) / t
            s["dentropy"] = _randn(g, t) * (0.05 / t) if case["entropy"] else None
            s["loss_scale"] = SCALE if case["type"] == "f16" else 1.0
            # the forward pass has been made: its row statistics are at hand
            s["saved"], s["entropy"] = _row_stats(s["x"], s["it"])
            s["entropy"] = s["entropy"] if case["entropy"] else None
    if own:
        _handles(s)
    return s


def _row_stats(x, it):
    """Row maximum and log of the row's sum, and the entropy, in chunks."""
    saved, ent = torch.empty(x.shape[0], 2, device="cuda"), torch.empty(x.shape[0], device="cuda")
    step = max(1, (1 << 26) // x.shape[1])
    for a in range(0, x.shape[0], step):
        r = x[a:a + step].float()
        top = r.amax(1)
        d = (r - top[:, None]) * it
        e = d.exp()
        tot = e.sum(1)
        saved[a:a + step, 0], saved[a:a + step, 1] = top, tot.log()
        ent[a:a + step] = tot.log() - torch.where(e > 0, e * d, 0.0).sum(1) / tot
    return saved, ent


def _handles(s):
    """What a program of the framework keeps between its calls: output buffers,
    the workspace, the control block and the list of tensors."""
    from zero_partitioned_mixed_partition_gb300 import binding as zs
    case, new = s["case"], lambda *n: torch.empty(*n, device="cuda")
    s["zs"], s["work"] = zs, zs.new_work()
    if "loss_scale" in s:
        s["ctrl"] = zs.new_ctrl()
        zs.zero_ctrl_init(s["ctrl"], s["loss_scale"])
    if case["op"] == "preference":
        s["out"] = {"loss": new(case["pairs"]), "reward": new(2 * case["pairs"]),
                    "totals": new(zs.ZS_PREFERENCE_TOTALS), "dlogp": new(s["n"])}
        s["hp"] = zs.preference(beta=s["beta"], kind=case["kind"], label_smoothing=0.1 if case["kind"] == "sigmoid" else 0.0,
                                margin=s["margin"], average=case["average"])
    elif case["op"] == "adamw":
        at = list(zip(s["offsets"], s["numels"]))
        part = lambda x, a, n: None if x is None else x[a:a + n]
        scale = lambda x, a, n: x[a // BLOCK:a // BLOCK + -(-n // BLOCK)] if case["state"] == 8 else None
        s["list"] = zs.TensorList([
            zs.TensorView(grad=part(s["grad"], a, n), master=part(s["master"], a, n), m=part(s["m"], a, n),
                          v=part(s["v"], a, n), param=part(s["copy"], a, n), m_scale=scale(s.get("m_scale"), a, n),
                          v_scale=scale(s.get("v_scale"), a, n), decay_mult=w)
            for (a, n), w in zip(at, s["decay"])])
        s["hp"] = zs.adam(LR, BETA1, BETA2, EPS, DECAY)
        s["sqnorm"] = zs.new_sqnorm()
        if case["state"] == 8:
            s["m_value"], s["v_value"] = new(s["n"]), new(s["n"])
    else:
        t = case["rows"]
        s["out"] = {"logp": new(t), "saved": new(t, 2), "entropy": new(t) if case["entropy"] else None}
        if case["op"] != "logp":
            s["out"]["dlogits"] = torch.empty(t, case["vocab"], dtype=s["x"].dtype, device="cuda")
        if case["op"] == "policy":
            s["out"]["token_loss"], s["out"]["totals"] = new(t), new(zs.ZS_POLICY_TOTALS)
            s["hp"] = zs.policy(**s["coef"])


# --------------------------------------------------------------- one pass ---

def run(s):
    return (_own if own else _plain)[s["case"]["op"]](s)


def _own_logp(s):
    o = s["out"]
    s["zs"].zero_token_logp_async(s["x"], s["labels"], o["logp"], entropy=o["entropy"], saved=o["saved"],
                                  inv_temperature=s["it"])
    return {"logp": o["logp"], "entropy": o["entropy"]}


def _own_logp_grad(s):
    s["zs"].zero_token_logp_grad_async(s["x"], s["labels"], s["saved"], s["dlogp"], s["out"]["dlogits"],
                                       entropy=s["entropy"], dentropy=s["dentropy"], inv_temperature=s["it"],
                                       ctrl_dev=s["ctrl"])
    return {"dlogits": s["out"]["dlogits"]}


def _own_policy(s):
    o = s["out"]
    s["zs"].zero_policy_loss_async(s["x"], s["labels"], s["old"], s["adv"], s["weights"], s["hp"], o["totals"],
                                   s["work"], ref_logp=s["ref"], logp=o["logp"], entropy=o["entropy"],
                                   token_loss=o["token_loss"], dlogits=o["dlogits"], inv_temperature=s["it"],
                                   ctrl_dev=s["ctrl"])
    return {k: o[k] for k in ("totals", "logp", "entropy", "token_loss", "dlogits")}


def _own_preference(s):
    o = s["out"]
    s["zs"].zero_preference_loss_async(s["logp"], s["cu"], s["hp"], o["loss"], o["reward"], o["totals"], s["work"],
                                       ref_logp=s["ref"], mask=s["mask"], dlogp=o["dlogp"])
    return o


def _own_adamw(s):
    zs, case = s["zs"], s["case"]
    zs.zero_tensors_sqnorm_async(s["list"], s["sqnorm"], s["work"], s["ctrl"])
    zs.zero_tensors_adamw_async(s["list"], s["hp"], s["ctrl"], max_norm=MAX_NORM if case["clip"] else 0.0,
                                sqnorm_dev=s["sqnorm"])
    out = {"sqnorm": s["sqnorm"].float(), "master": s["master"], "copy": s["copy"]}
    if case["state"] == 32:
        return {**out, "m": s["m"], "v": s["v"]}
    # the 8-bit states as the values that they stand for
    zs.zero_adam8_dequantize(s["m"], s["m_scale"], s["n"], True, s["m_value"])
    zs.zero_adam8_dequantize(s["v"], s["v_scale"], s["n"], False, s["v_value"])
    return {**out, "m": s["m_value"], "v": s["v_value"]}


_own = {"logp": _own_logp, "logp_grad": _own_logp_grad, "policy": _own_policy, "preference": _own_preference,
        "adamw": _own_adamw}


def _plain_rows(s, valid):
    """Of every row: shifted logits, their exponentials and sum, log-probability
    of the label, entropy; rows that are not valid give zeros."""
    x, it = s["x"].float(), s["it"]
    y = s["labels"].clamp(min=0)[:, None]
    d = (x - x.amax(1, keepdim=True)) * it
    del x
    e = d.exp()
    tot = e.sum(1, keepdim=True)
    zero = torch.zeros((), device="cuda")
    logp = torch.where(valid, (d.gather(1, y) - tot.log())[:, 0], zero)
    ent = None
    if s["case"]["entropy"]:
        ent = torch.where(valid, (tot.log() - torch.where(e > 0, e * d, zero).sum(1, keepdim=True) / tot)[:, 0], zero)
    return d, e, tot, y, logp, ent


def _plain_dlogits(s, rows, valid, dlogp, dent):
    d, e, tot, y, _, ent = rows
    p = e / tot
    dx = p * -dlogp[:, None]
    dx.scatter_add_(1, y, dlogp[:, None])
    if dent is not None:
        dx -= dent[:, None] * torch.where(e > 0, p * (d - tot.log() + ent[:, None]), torch.zeros((), device="cuda"))
    dx *= s["it"] * s["loss_scale"]
    dx.masked_fill_(~valid[:, None], 0.0)
    return dx.to(s["x"].dtype)


def _plain_logp(s):
    valid = s["labels"] >= 0
    _, _, _, _, logp, ent = _plain_rows(s, valid)
    return {"logp": logp, "entropy": ent}


def _plain_logp_grad(s):
    valid = s["labels"] >= 0
    d = (s["x"].float() - s["saved"][:, :1]) * s["it"]
    tot = s["saved"][:, 1:].exp()
    rows = (d, d.exp(), tot, s["labels"].clamp(min=0)[:, None], None, s["entropy"])
    return {"dlogits": _plain_dlogits(s, rows, valid, s["dlogp"], s["dentropy"])}


def _plain_policy(s):
    c, w = s["coef"], s["weights"]
    valid = w != 0
    rows = _plain_rows(s, valid)
    logp, ent = rows[4], rows[5]
    zero = torch.zeros((), device="cuda")
    ratio = (logp - s["old"]).exp()
    held = ratio.clamp(1.0 - c["clip_low"], 1.0 + c["clip_high"])
    free, bound = -s["adv"] * ratio, -s["adv"] * held
    clipped = free < bound
    pg = torch.maximum(free, bound)
    dpg = torch.where(clipped, zero, free)
    capped = (s["adv"] < 0) & (pg > -s["adv"] * c["dual_clip"])
    pg = torch.where(capped, -s["adv"] * c["dual_clip"], pg)
    dpg = torch.where(capped, zero, dpg)
    gap = s["ref"] - logp
    kl = gap.exp() - gap - 1.0
    loss = pg + c["kl_coef"] * kl
    if ent is not None:
        loss = loss - c["entropy_coef"] * ent
    dlogp = torch.where(valid, w * (dpg + c["kl_coef"] * (1.0 - gap.exp())), zero)
    dent = -c["entropy_coef"] * w if ent is not None else None
    token = torch.where(valid, loss, zero)
    sums = [token, torch.where(valid, pg, zero), torch.where(valid, kl, zero), zero * w if ent is None else ent,
            (valid & (clipped | capped)).float()]
    return {"totals": (torch.stack(sums) * w).sum(1), "logp": logp, "entropy": ent, "token_loss": token,
            "dlogits": _plain_dlogits(s, rows, valid, dlogp, dent)}


def _plain_preference(s):
    case, mask = s["case"], s["mask"]
    p, beta, zero = case["pairs"], s["beta"], torch.zeros((), device="cuda")
    # the sequences side by side, filled up to the longest
    at = s["cu"][:-1, None] + torch.arange(s["longest"], device="cuda")
    inside = at < s["cu"][1:, None]
    at.clamp_(max=max(0, s["n"] - 1))
    inside &= mask[at]
    diff = (s["logp"] - s["ref"] if case["ref"] else s["logp"])[at]
    total = torch.where(inside, diff, zero).sum(1)
    count = inside.float().sum(1)
    del at, inside, diff
    share = 1.0 / count.clamp(min=1.0) if case["average"] else torch.ones(2 * p, device="cuda")
    score = total * share
    h = score[0::2] - score[1::2]
    z = beta * h - s["margin"]
    if case["kind"] == "sigmoid":
        soft = lambda u: torch.clamp(u, min=0.0) + (1.0 + (-u.abs()).exp()).log()
        loss = 0.9 * soft(-z) + 0.1 * soft(z)
        dz = 0.1 / (1.0 + (-z).exp()) - 0.9 / (1.0 + z.exp())
        dh = beta * dz
    elif case["kind"] == "hinge":
        loss = (1.0 - z).clamp(min=0.0)
        dh = torch.where(z < 1.0, -beta, 0.0)
    else:
        loss = (h - 1.0 / (2.0 * beta)).square()
        dh = 2.0 * (h - 1.0 / (2.0 * beta))
    reward = beta * score
    win = (reward[0::2] > reward[1::2]).float()
    totals = torch.stack([loss, win, reward[0::2] - reward[1::2]]).sum(1) / p
    each = torch.stack([dh, -dh], 1).reshape(-1) * share / p
    seq = torch.repeat_interleave(torch.arange(2 * p, device="cuda"), s["cu"][1:] - s["cu"][:-1], output_size=s["n"])
    return {"loss": loss, "reward": reward, "totals": totals, "dlogp": torch.where(mask, each[seq], zero)}


def _map(bits):
    """Values of the 8-bit states' map with `bits` bits, in 32 bits."""
    out = [0.0]
    for k in range(1, 1 << bits):
        f = k.bit_length() - 1
        out.append((0.1 + 0.9 * ((k - (1 << f) + 1) / (1 << f))) / 10.0 ** (bits - f - 1))
    return torch.tensor(out, dtype=torch.float32)


_maps = {}


def _tables(bits):
    """The map, and for each pair of neighbours the largest float not above
    their midpoint: a value above it is nearer to the upper one."""
    if bits not in _maps:
        m = _map(bits).double()
        mid = (m[1:] + m[:-1]) / 2
        t = mid.float()
        t = torch.where(t.double() > mid, torch.nextafter(t, torch.zeros(())), t)
        _maps[bits] = (m.float().cuda(), t.cuda())
    return _maps[bits]


def _decode(codes, scale, signed):
    code = codes.int()
    value = _tables(7 if signed else 8)[0][code & 127 if signed else code]
    if signed:
        value = torch.where(code >= 128, -value, value)
    return (value.view(-1, BLOCK) * scale[:, None]).view(-1)


def _encode(value, codes, scale, signed):
    """Quantizes in place and returns what the codes stand for."""
    top = value.view(-1, BLOCK).abs().amax(1)
    scale.copy_(top)
    x = (value.view(-1, BLOCK) / torch.where(top > 0, top, torch.ones((), device="cuda"))[:, None]).view(-1)
    code = torch.bucketize(x.abs(), _tables(7 if signed else 8)[1], out_int32=True)
    if signed:
        code = torch.where((x < 0) & (code > 0), code + 128, code)
    codes.copy_(code)
    del x, code
    return _decode(codes, scale, signed)


def _plain_adamw(s):
    case = s["case"]
    s["beta_pow"] = [s["beta_pow"][0] * BETA1, s["beta_pow"][1] * BETA2]
    bc1, bc2 = 1.0 - s["beta_pow"][0], 1.0 - s["beta_pow"][1]
    g = s["grad"].float() * (1.0 / s["loss_scale"])
    sq = (g * g).sum()
    if case["clip"]:
        g = g * torch.clamp(MAX_NORM / (sq.sqrt() + 1e-6), max=1.0)
    small = case["state"] == 8
    m = _decode(s["m"], s["m_scale"], True) if small else s["m"]
    m = m * BETA1 + g * (1.0 - BETA1)
    v = _decode(s["v"], s["v_scale"], False) if small else s["v"]
    v = v * BETA2 + (g * g) * (1.0 - BETA2)
    del g
    u = (m / bc1) / ((v / bc2).sqrt() + EPS)
    decay = torch.tensor([DECAY * w for w in s["decay"]], device="cuda")
    decay = torch.repeat_interleave(decay, s["spans"], output_size=s["n"])
    s["master"].sub_((u + decay * s["master"]) * LR)
    del u, decay
    if s["copy"] is not None:
        s["copy"].copy_(s["master"])
    if small:
        m = _encode(m, s["m"], s["m_scale"], True)
        v = _encode(v, s["v"], s["v_scale"], False)
    else:
        s["m"].copy_(m)
        s["v"].copy_(v)
        m, v = s["m"], s["v"]
    return {"sqnorm": sq.view(1), "master": s["master"], "copy": s["copy"], "m": m, "v": v}


_plain = {"logp": _plain_logp, "logp_grad": _plain_logp_grad, "policy": _plain_policy, "preference": _plain_preference,
          "adamw": _plain_adamw}


# ------------------------------------------------------------ what it costs ---

def work(case):
    if case["op"] == "preference":
        n = 2 * case["pairs"] * case["mean"]
        return {"bytes": n * (4 + 1 + 4 + (4 if case["ref"] else 0)) + 36 * case["pairs"], "flops": 4 * n}
    if case["op"] == "adamw":
        n = sum(_numels(case))
        copy = 0 if case["copy"] == "none" else SIZE[case["copy"]]
        # gradient, weights (in and out), copy, states (in and out; 8-bit ones come back as values too)
        return {"bytes": n * (SIZE[case["type"]] + 8 + copy + (16 if case["state"] == 32 else 12)), "flops": 16 * n}
    t, v, size = case["rows"], case["vocab"], SIZE[case["type"]]
    reads = t * (1.0 - case["ignored"]) * v * size
    if case["op"] == "logp":
        return {"bytes": reads + t * (8 + 4 + (4 if case["entropy"] else 0)), "flops": 4 * t * v}
    return {"bytes": reads + t * v * size + t * 40, "flops": 8 * t * v}


# ---------------------------------------------------------------- 64 bits ---

def exact(case, seed):
    with torch.enable_grad():
        s = _without_own(case, seed)
        if case["op"] == "preference":
            return _exact_preference(s)
        if case["op"] == "adamw":
            return _exact_adamw(s)
        return _exact_rows(s)


def _without_own(case, seed):
    global own
    was, own = own, False
    try:
        return prepare(case, seed)
    finally:
        own = was


def _exact_rows(s):
    """The definition on torch.double rows, gradients by differentiation, some
    rows at a time."""
    case, t, v = s["case"], s["case"]["rows"], s["case"]["vocab"]
    f64 = lambda *n: torch.zeros(*n, dtype=torch.float64, device="cuda")
    policy, back = case["op"] == "policy", case["op"] != "logp"
    valid = s["weights"] != 0 if policy else s["labels"] >= 0
    out = {"logp": f64(t), "entropy": f64(t) if case["entropy"] else None}
    if back:
        out["dlogits"] = f64(t, v)
    if policy:
        out["token_loss"], out["totals"] = f64(t), f64(5)
    step = max(1, (1 << 25) // v)
    for a in range(0, t, step):
        rows = torch.nonzero(valid[a:a + step])[:, 0] + a
        if not len(rows):
            continue
        x = s["x"][rows].double().requires_grad_(back)
        lp = torch.log_softmax(x / case["temperature"], 1)
        logp = lp[torch.arange(len(rows), device="cuda"), s["labels"][rows]]
        ent = -(lp.exp() * lp.masked_fill(torch.isinf(lp), 0.0)).sum(1) if case["entropy"] else None
        out["logp"][rows] = logp.detach()
        if ent is not None:
            out["entropy"][rows] = ent.detach()
        if case["op"] == "logp_grad":
            (logp * s["dlogp"][rows]).sum().add(0.0 if ent is None else (ent * s["dentropy"][rows]).sum()).backward()
        elif policy:
            c, w, adv = s["coef"], s["weights"][rows].double(), s["adv"][rows].double()
            r = (logp - s["old"][rows].double()).exp()
            lo, hi = 1.0 - c["clip_low"], 1.0 + c["clip_high"]
            pg = -torch.minimum(adv * r, adv * r.clamp(lo, hi))
            off = adv * r > adv * r.clamp(lo, hi)
            cap = (adv < 0) & (pg > -c["dual_clip"] * adv)
            pg = torch.where(cap, -c["dual_clip"] * adv, pg)
            gap = s["ref"][rows].double() - logp
            kl = gap.exp() - 1.0 - gap
            loss = pg + c["kl_coef"] * kl - (0.0 if ent is None else c["entropy_coef"] * ent)
            out["token_loss"][rows] = loss.detach()
            ones = [loss, pg, kl, torch.zeros_like(kl) if ent is None else ent, (off | cap).double()]
            out["totals"] += torch.stack([(w * o.detach()).sum() for o in ones])
            (w * loss).sum().backward()
        if back:
            out["dlogits"][rows] = x.grad * s["loss_scale"]
        del x, lp
    if case["op"] == "logp_grad":
        return {"dlogits": out["dlogits"]}
    return out


def _exact_preference(s):
    case, p = s["case"], s["case"]["pairs"]
    logp = s["logp"].double().requires_grad_(True)
    diff = (logp - (s["ref"].double() if case["ref"] else 0.0)) * s["mask"]
    seq = torch.bucketize(torch.arange(s["n"], device="cuda"), s["cu"][1:], right=True)
    score = torch.zeros(2 * p, dtype=torch.float64, device="cuda").index_add(0, seq, diff)
    if case["average"]:
        score = score / torch.zeros_like(score).index_add(0, seq, s["mask"].double()).clamp(min=1.0)
    h = score.view(p, 2)[:, 0] - score.view(p, 2)[:, 1]
    z = s["beta"] * h - s["margin"]
    logsig = torch.nn.functional.logsigmoid
    loss = {"sigmoid": lambda: -0.9 * logsig(z) - 0.1 * logsig(-z), "hinge": lambda: torch.relu(1.0 - z),
            "squared": lambda: (h - 0.5 / s["beta"]) ** 2}[case["kind"]]()
    loss.mean().backward()
    reward = (s["beta"] * score).detach()
    gain = reward.view(p, 2)[:, 0] - reward.view(p, 2)[:, 1]
    return {"loss": loss.detach(), "reward": reward, "totals": torch.stack([loss.detach().mean(), (gain > 0).double().mean(), gain.mean()]),
            "dlogp": logp.grad}


def _exact_adamw(s):
    case, small = s["case"], s["case"]["state"] == 8
    sq = torch.zeros(1, dtype=torch.float64, device="cuda")
    step = 1 << 26
    for a in range(0, s["n"], step):
        sq += (s["grad"][a:a + step].double() / s["loss_scale"]).square().sum()
    clip = min(1.0, MAX_NORM / (math.sqrt(sq.item()) + 1e-6)) if case["clip"] else 1.0
    out = {k: torch.zeros(s["n"], dtype=torch.float64, device="cuda") for k in ("master", "m", "v")}
    for at, n, w in zip(s["offsets"], s["numels"], s["decay"]):
        for a in range(at, at + n, step):
            b = min(at + n, a + step)
            g = s["grad"][a:b].double() * (clip / s["loss_scale"])
            old = {}
            for k, bits in (("m", 7), ("v", 8)):
                if small:
                    code = s[k][a:b].long()
                    value = _map(bits).double().cuda()[code % 128 if k == "m" else code]
                    value = value * torch.where(code > 127, -1.0, 1.0) if k == "m" else value
                    old[k] = value * s[k + "_scale"][a // BLOCK:-(-b // BLOCK)].double().repeat_interleave(BLOCK)[:b - a]
                else:
                    old[k] = s[k][a:b].double()
            m = BETA1 * old["m"] + (1.0 - BETA1) * g
            v = BETA2 * old["v"] + (1.0 - BETA2) * g * g
            th = s["master"][a:b].double()
            u = (m / (1.0 - BETA1)) / ((v / (1.0 - BETA2)).sqrt() + EPS)
            out["master"][a:b] = th - LR * (u + DECAY * w * th)
            out["m"][a:b] = _nearest(m, 7) if small else m
            out["v"][a:b] = _nearest(v, 8) if small else v
    return {"sqnorm": sq, "master": out["master"], "copy": None if s["copy"] is None else out["master"], "m": out["m"], "v": out["v"]}


def _nearest(value, bits):
    """Each block's values replaced by the nearest multiples of the map."""
    table = _map(bits).double().cuda()
    whole = torch.nn.functional.pad(value, (0, -len(value) % BLOCK)).view(-1, BLOCK)
    top = whole.abs().max(1, keepdim=True).values
    x = whole.abs() / top.clamp(min=1e-300)
    up = torch.searchsorted(table, x.contiguous()).clamp(1, len(table) - 1)
    lower, upper = table[up - 1], table[up]
    near = torch.where(x - lower <= upper - x, lower, upper)
    return (near * top * whole.sign()).view(-1)[:len(value)]
