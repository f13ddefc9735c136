"""Workloads of a language model's two ends: token log-probabilities straight
from hidden states and the vocabulary matrix (the logits are never kept), layer
norm, and the embedding lookup, each with its gradient.

``listed()`` and ``draw()`` name the cases, ``prepare()`` makes a case's inputs
on the GPU, ``run()`` makes one pass: with ``own`` the calls of the framework,
otherwise the same operator in elementary 32-bit torch operations.
``exact()`` is the definition in 64 bits.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
SCALE = 1024.0                     # loss scale carried by fp16 gradients
MOST_FLOPS = 2.0e13                # of a drawn head
MOST_NUMEL = 1 << 27               # of a drawn norm's or embedding's rows


# ------------------------------------------------------------------- cases ---

def listed():
    return [
        # scoring the four sequences' current tokens: the vocabulary matrix is read for four rows
        {"name": "head logp small", "op": "head", "rows": 4, "vocab": 32000, "width": 4096, "type": "bf16",
         "ignored": 0.0, "temperature": 0.7},
        # scoring a packed batch of the small model; prompts ignored
        {"name": "head logp batch", "op": "head", "rows": 8192, "vocab": 50257, "width": 768, "type": "bf16",
         "ignored": 0.25, "temperature": 1.0},
        # backward of a micro-batch of a 1600 wide model
        {"name": "head gradient batch", "op": "head_grad", "rows": 2048, "vocab": 50257, "width": 1600, "type": "f16",
         "ignored": 0.3, "temperature": 1.0},
        # backward of a large micro-batch over a large vocabulary: several pieces of the vocabulary
        {"name": "head gradient large", "op": "head_grad", "rows": 8192, "vocab": 131072, "width": 4096, "type": "bf16",
         "ignored": 0.1, "temperature": 1.0},
        # the final norm of a few tokens: latency
        {"name": "norm small", "op": "norm", "rows": 16, "width": 768, "type": "f32", "params": "f32"},
        # the norm of a packed batch
        {"name": "norm batch", "op": "norm", "rows": 16384, "width": 1600, "type": "bf16", "params": "bf16"},
        # backward of an odd width in fp16 (adapters' and vision widths are not all multiples of eight)
        {"name": "norm gradient odd", "op": "norm_grad", "rows": 1777, "width": 1001, "type": "f16", "params": "f32"},
        # backward of a large batch of a wide model
        {"name": "norm gradient large", "op": "norm_grad", "rows": 16384, "width": 4096, "type": "bf16", "params": "f32"},
        # the next tokens of eight sequences: latency
        {"name": "embed small", "op": "embed", "tokens": 8, "vocab": 50257, "width": 768, "type": "f16", "scale": 1.0},
        # a long packed batch, rows scaled by the root of the width
        {"name": "embed batch", "op": "embed", "tokens": 65536, "vocab": 32000, "width": 4096, "type": "bf16", "scale": 64.0},
        # gradient of the table of the small model: most rows get nothing, a few tokens come hundreds of times
        {"name": "embed gradient batch", "op": "embed_grad", "tokens": 8192, "vocab": 50257, "width": 768, "type": "bf16",
         "grad": "bf16", "scale": 1.0, "add": False},
        # a tied table: added to the gradient that the head left there, kept in fp32
        {"name": "embed gradient tied", "op": "embed_grad", "tokens": 65536, "vocab": 32000, "width": 4096, "type": "bf16",
         "grad": "f32", "scale": 64.0, "add": True},
    ]


def _log_between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["head", "head_grad", "head_grad", "norm", "norm_grad", "embed", "embed_grad", "embed_grad"])
    kind = rng.choice(["bf16", "f16"])
    if op in ("head", "head_grad"):
        vocab, width = _log_between(rng, 500, 200_000), 8 * _log_between(rng, 8, 512)
        most = MOST_FLOPS / ((2.0 if op == "head" else 6.0) * vocab * width)
        return {"op": op, "rows": _log_between(rng, 1, max(1, min(12_000, int(most)))), "vocab": vocab, "width": width,
                "type": kind, "ignored": rng.choice([0.0, 0.3, 0.8]), "temperature": rng.choice([1.0, 0.7, 1.3])}
    width = _log_between(rng, 30, 8192)
    if rng.random() < 0.6:
        width = max(8, width // 8 * 8)
    rows = _log_between(rng, 1, min(65536, MOST_NUMEL // (2 * width)))
    if op in ("norm", "norm_grad"):
        kind = rng.choice(["bf16", "f16", "f32"])
        return {"op": op, "rows": rows, "width": width, "type": kind, "params": rng.choice([kind, "f32"])}
    kind = rng.choice(["bf16", "f16", "f32"])
    case = {"op": op, "tokens": rows, "vocab": _log_between(rng, 100, min(200_000, MOST_NUMEL // width)), "width": width,
            "type": kind, "scale": rng.choice([1.0, 0.7, 12.5])}
    if op == "embed_grad":
        case.update({"grad": rng.choice([kind, "f32"]), "add": rng.random() < 0.4})
        if case["add"] and case["grad"] == "f16":
            case["grad"] = "f32"       # sums that grow from pass to pass would leave fp16's range
    return case


# ------------------------------------------------------------------ inputs ---

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda")


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _matrix(g, rows, width, kind, spread):
    """Normal values, made in parts."""
    out = torch.empty(rows, width, dtype=TYPES[kind], device="cuda")
    step = max(1, (1 << 26) // width)
    for a in range(0, rows, step):
        out[a:a + step] = _randn(g, min(step, rows - a), width) * spread
    return out


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case, "loss_scale": SCALE if case["type"] == "f16" else 1.0}
    if case["op"] in ("head", "head_grad"):
        n, v, d = case["rows"], case["vocab"], case["width"]
        s["it"] = 1.0 / case["temperature"]
        # logits of spread 2.5 in which each row's label stands out by 0 to 9
        s["weight"] = _matrix(g, v, d, case["type"], 2.5 / math.sqrt(d))
        s["labels"] = torch.randint(0, v, (n,), generator=g, device="cuda")
        boost = _rand(g, n, 1) * (9.0 / 6.25)
        s["hidden"] = (_randn(g, n, d) + boost * s["weight"][s["labels"]].float()).to(TYPES[case["type"]])
        skip = _rand(g, n) < case["ignored"]
        s["labels"] = torch.where(skip, torch.full_like(s["labels"], -100), s["labels"])
        if case["op"] == "head_grad":
            # the weights of a policy's or a pair's tokens, either sign
            s["dlogp"] = _randn(g, n) / n
            # the forward pass has been made: its row statistics are at hand
            s["saved"] = _saved(s)
    elif case["op"] in ("norm", "norm_grad"):
        n, d = case["rows"], case["width"]
        s["x"] = (_randn(g, n, d) * (0.5 + 3.0 * _rand(g, n, 1)) + _randn(g, n, 1)).to(TYPES[case["type"]])
        s["gamma"] = (1.0 + 0.2 * _randn(g, d)).to(TYPES[case["params"]])
        s["beta"] = (0.2 * _randn(g, d)).to(TYPES[case["params"]])
        s["eps"] = 1e-5
        if case["op"] == "norm_grad":
            s["dy"] = _matrix(g, n, d, case["type"], s["loss_scale"] / n)
            s["saved"] = _norm_stats(s["x"].float(), s["eps"])
    else:
        n, v, d = case["tokens"], case["vocab"], case["width"]
        # frequencies that fall as one over the rank; the ranks lie anywhere in the vocabulary
        rank = ((_rand(g, n).double() * math.log(v + 1)).exp().long() - 1).clamp(0, v - 1)
        s["ids"] = torch.randperm(v, generator=g, device="cuda")[rank]
        if case["op"] == "embed":
            s["table"] = _matrix(g, v, d, case["type"], 0.02)
        else:
            s["dout"] = _matrix(g, n, d, case["type"], s["loss_scale"] * 1e-3)
            s["dtable"] = _matrix(g, v, d, case["grad"], s["loss_scale"] * 1e-2) if case["add"] else \
                torch.empty(v, d, dtype=TYPES[case["grad"]], device="cuda")
    if own:
        _handles(s)
    return s


def _saved(s):
    """A row's largest logit and the log of its sum, in parts of the rows."""
    h, w = s["hidden"], s["weight"].float()
    out = torch.empty(h.shape[0], 2, device="cuda")
    step = max(1, (1 << 28) // w.shape[0])
    for a in range(0, h.shape[0], step):
        x = h[a:a + step].float() @ w.t()
        out[a:a + step, 0] = x.amax(1)
        out[a:a + step, 1] = ((x - out[a:a + step, :1]) * s["it"]).exp().sum(1).log()
    return out


def _norm_stats(x, eps):
    mean = x.mean(1, keepdim=True)
    return torch.cat([mean, ((x - mean).square().mean(1, keepdim=True) + eps).rsqrt()], 1)


def _handles(s):
    """What a program of the framework keeps between its calls: output buffers,
    the workspace and the control block."""
    from zero_partitioned_mixed_partition_gb300 import binding as zs
    case, new = s["case"], lambda *n: torch.empty(*n, device="cuda")
    s["zs"] = zs
    if case["op"] in ("head", "head_grad"):
        n = case["rows"]
        s["work"] = zs.new_head_work(n, case["width"], case["vocab"], gradient=case["op"] == "head_grad")
        if case["op"] == "head":
            s["out"] = {"logp": new(n), "saved": new(n, 2)}
        else:
            s["ctrl"] = zs.new_ctrl()
            zs.zero_ctrl_init(s["ctrl"], s["loss_scale"])
            s["out"] = {"dhidden": torch.empty_like(s["hidden"]), "dweight": torch.empty_like(s["weight"])}
    elif case["op"] == "norm":
        s["out"] = {"y": torch.empty_like(s["x"]), "saved": new(case["rows"], 2)}
    elif case["op"] == "norm_grad":
        s["work"] = zs.new_layer_norm_work(case["rows"], case["width"])
        s["out"] = {"dx": torch.empty_like(s["x"]), "dgamma": torch.empty_like(s["gamma"]),
                    "dbeta": torch.empty_like(s["beta"])}
    elif case["op"] == "embed":
        s["out"] = torch.empty(case["tokens"], case["width"], dtype=s["table"].dtype, device="cuda")
    else:
        s["work"] = zs.new_embed_work(case["tokens"], case["width"])


# --------------------------------------------------------------- one pass ---

def run(s):
    return (_own if own else _plain)[s["case"]["op"]](s)


def _own_head(s):
    o = s["out"]
    s["zs"].zero_head_logp_async(s["hidden"], s["weight"], s["labels"], o["logp"], s["work"], saved=o["saved"],
                                 inv_temperature=s["it"])
    return o


def _own_head_grad(s):
    o = s["out"]
    s["zs"].zero_head_logp_grad_async(s["hidden"], s["weight"], s["labels"], s["saved"], s["dlogp"], o["dhidden"],
                                      o["dweight"], s["work"], inv_temperature=s["it"], ctrl_dev=s["ctrl"])
    return o


def _own_norm(s):
    o = s["out"]
    s["zs"].zero_layer_norm_async(s["x"], s["gamma"], s["beta"], o["y"], saved=o["saved"], eps=s["eps"])
    return o


def _own_norm_grad(s):
    o = s["out"]
    s["zs"].zero_layer_norm_grad_async(s["dy"], s["x"], s["gamma"], s["saved"], o["dx"], o["dgamma"], o["dbeta"],
                                       s["work"])
    return o


def _own_embed(s):
    s["zs"].zero_embed_async(s["table"], s["ids"], s["out"], scale=s["case"]["scale"])
    return {"out": s["out"]}


def _own_embed_grad(s):
    s["zs"].zero_embed_grad_async(s["ids"], s["dout"], s["dtable"], s["work"], scale=s["case"]["scale"],
                                  accumulate=s["case"]["add"])
    return {"dtable": s["dtable"]}


_own = {"head": _own_head, "head_grad": _own_head_grad, "norm": _own_norm, "norm_grad": _own_norm_grad,
        "embed": _own_embed, "embed_grad": _own_embed_grad}


def _plain_head(s):
    valid = s["labels"] >= 0
    x = s["hidden"].float() @ s["weight"].float().t()
    top, zero = x.amax(1, keepdim=True), torch.zeros((), device="cuda")
    d = (x - top) * s["it"]
    total = d.exp().sum(1, keepdim=True).log()
    logp = (d.gather(1, s["labels"].clamp(min=0)[:, None]) - total)[:, 0]
    return {"logp": torch.where(valid, logp, zero), "saved": torch.where(valid[:, None], torch.cat([top, total], 1), zero)}


def _plain_head_grad(s):
    valid = s["labels"] >= 0
    h, w = s["hidden"].float(), s["weight"].float()
    x = h @ w.t()
    p = ((x - s["saved"][:, :1]) * s["it"] - s["saved"][:, 1:]).exp()
    c = torch.where(valid, s["dlogp"], torch.zeros((), device="cuda")) * (s["it"] * s["loss_scale"])
    dl = p * -c[:, None]
    dl.scatter_add_(1, s["labels"].clamp(min=0)[:, None], c[:, None])
    del x, p
    return {"dhidden": (dl @ w).to(s["hidden"].dtype), "dweight": (dl.t() @ h).to(s["weight"].dtype)}


def _plain_norm(s):
    x = s["x"].float()
    saved = _norm_stats(x, s["eps"])
    y = (x - saved[:, :1]) * saved[:, 1:] * s["gamma"].float() + s["beta"].float()
    return {"y": y.to(s["x"].dtype), "saved": saved}


def _plain_norm_grad(s):
    x, dy = s["x"].float(), s["dy"].float()
    xh = (x - s["saved"][:, :1]) * s["saved"][:, 1:]
    a = dy * s["gamma"].float()
    dx = s["saved"][:, 1:] * (a - a.mean(1, keepdim=True) - xh * (a * xh).mean(1, keepdim=True))
    return {"dx": dx.to(s["x"].dtype), "dgamma": (dy * xh).sum(0).to(s["gamma"].dtype),
            "dbeta": dy.sum(0).to(s["beta"].dtype)}


def _plain_embed(s):
    return {"out": (s["table"][s["ids"]].float() * s["case"]["scale"]).to(s["table"].dtype)}


def _plain_embed_grad(s):
    # one sum for each token of the vocabulary: the frequent ones add up thousands of rows
    total = torch.zeros(s["dtable"].shape, device="cuda")
    total.index_add_(0, s["ids"], s["dout"].float())
    total *= s["case"]["scale"]
    if s["case"]["add"]:
        total += s["dtable"].float()
    s["dtable"].copy_(total)
    return {"dtable": s["dtable"]}


_plain = {"head": _plain_head, "head_grad": _plain_head_grad, "norm": _plain_norm, "norm_grad": _plain_norm_grad,
          "embed": _plain_embed, "embed_grad": _plain_embed_grad}


# ------------------------------------------------------------------- work ---

def _distinct(tokens, vocab):
    """Expected number of different tokens among `tokens`."""
    r = torch.arange(1, vocab + 1, dtype=torch.float64)
    p = ((r + 1).log() - r.log()) / math.log(vocab + 1)
    return float((1.0 - (1.0 - p) ** tokens).sum())


def work(case):
    size, op = SIZE[case["type"]], case["op"]
    if op in ("head", "head_grad"):
        n, v, d = case["rows"], case["vocab"], case["width"]
        live = (1.0 - case["ignored"]) * n
        if op == "head":
            return {"bytes": (live + v) * d * size + 20 * n, "flops": 2.0 * live * v * d}
        return {"bytes": (live + n + 2 * v) * d * size + 20 * n, "flops": 6.0 * live * v * d}
    if op in ("norm", "norm_grad"):
        n, d, p = case["rows"], case["width"], SIZE[case["params"]]
        if op == "norm":
            return {"bytes": 2 * n * d * size + 2 * d * p + 8 * n, "flops": 8.0 * n * d}
        return {"bytes": 3 * n * d * size + 3 * d * p + 8 * n, "flops": 14.0 * n * d}
    n, v, d = case["tokens"], case["vocab"], case["width"]
    if op == "embed":
        return {"bytes": (n + _distinct(n, v)) * d * size + 8 * n, "flops": 1.0 * n * d}
    g = SIZE[case["grad"]]
    table = 2 * _distinct(n, v) if case["add"] else v
    return {"bytes": n * d * size + table * d * g + 8 * n, "flops": 1.0 * n * d}


# ------------------------------------------------------------------- exact ---

def exact(case, seed):
    """The operators' definition in 64 bits on the inputs of prepare(case, seed)."""
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    f64 = torch.float64
    if case["op"] in ("head", "head_grad"):
        n, v, d = case["rows"], case["vocab"], case["width"]
        if (2.0 if case["op"] == "head" else 6.0) * n * v * d > 5e12:
            return None
        h, w, y = s["hidden"].to(f64), s["weight"].to(f64), s["labels"]
        live = (y >= 0).nonzero()[:, 0]
        logp, saved = torch.zeros(n, dtype=f64, device="cuda"), torch.zeros(n, 2, dtype=f64, device="cuda")
        dh, dw = torch.zeros_like(h), torch.zeros_like(w)
        step = max(1, (1 << 27) // v)
        for a in range(0, len(live), step):
            i = live[a:a + step]
            x = h[i] @ w.T
            lp = torch.log_softmax(x / case["temperature"], 1)
            if case["op"] == "head":
                logp[i] = lp[torch.arange(len(i), device="cuda"), y[i]]
                saved[i, 0] = x.max(1).values
                saved[i, 1] = torch.logsumexp(x / case["temperature"], 1) - saved[i, 0] / case["temperature"]
                continue
            e = -lp.exp()
            e[torch.arange(len(i), device="cuda"), y[i]] += 1.0
            e *= (s["dlogp"][i].to(f64) * (s["loss_scale"] / case["temperature"]))[:, None]
            dh[i] = e @ w
            dw += e.T @ h[i]
        return {"logp": logp, "saved": saved} if case["op"] == "head" else {"dhidden": dh, "dweight": dw}
    if case["op"] in ("norm", "norm_grad"):
        x, gamma, beta = s["x"].to(f64), s["gamma"].to(f64), s["beta"].to(f64)
        mu = x.mean(1)
        r = 1.0 / torch.sqrt(x.var(1, unbiased=False) + s["eps"])
        z = (x - mu[:, None]) * r[:, None]
        if case["op"] == "norm":
            return {"y": z * gamma + beta, "saved": torch.stack([mu, r], 1)}
        dy = s["dy"].to(f64)
        a, d = dy * gamma, case["width"]
        dx = (d * a - a.sum(1)[:, None] - z * (a * z).sum(1)[:, None]) * (r / d)[:, None]
        return {"dx": dx, "dgamma": torch.einsum("nd,nd->d", dy, z), "dbeta": dy.sum(0)}
    if case["op"] == "embed":
        return {"out": s["table"].to(f64).index_select(0, s["ids"]) * case["scale"]}
    # rows in the order of their tokens, then one segment after the other
    order = torch.argsort(s["ids"], stable=True)
    ids, count = torch.unique_consecutive(s["ids"][order], return_counts=True)
    ends = count.cumsum(0)
    out = s["dtable"].to(f64) if case["add"] else torch.zeros(s["dtable"].shape, dtype=f64, device="cuda")
    step = max(1, (1 << 27) // case["tokens"])
    for a in range(0, case["width"], step):
        run_sum = s["dout"][:, a:a + step].to(f64)[order].cumsum(0)[ends - 1]
        run_sum[1:] -= run_sum[:-1].clone()
        out[ids, a:a + step] += run_sum * case["scale"]
    return {"dtable": out}
