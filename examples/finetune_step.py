"""Fine-tuning steps of a small language model on one GPU with the library's
loss and tensor-list calls: supervised by rewards (the clipped policy loss), by
pairs (the preference loss) or by the next token itself (cross entropy), each step ended by AdamW
over the model's tensors.

    python examples/finetune_step.py [--steps 30] [--loss policy|preference|supervised]

The model predicts the next token from the last one: logits = gelu(E[token] + b)
W^T, weights in bf16 with fp32 masters.  A step runs

    scoring      zero_token_logp_async (old and reference log-probabilities)
    loss         zero_policy_loss_async, or zero_preference_loss_async and
                 zero_token_logp_grad_async: the loss-scaled gradient of the logits
    backward     plain torch products
    optimizer    zero_tensors_sqnorm_async, zero_tensors_adamw_async: unscaled,
                 clipped, skipped on the device if a gradient overflowed; the two
                 matrices keep 8-bit states, the bias fp32 ones

and nothing in it waits for the GPU but the printed line.

With --loss supervised the model is logits = LN(E[token]) E^T, its two ends tied, and every
part of the step is a call of the library; the logits are never kept:

    forward      zero_embed_async, zero_layer_norm_async, zero_head_logp_async
    backward     zero_head_logp_grad_async, zero_layer_norm_grad_async, and
                 zero_embed_grad_async added to the head's gradient of E
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from zero_partitioned_mixed_partition_gb300 import binding as zs  # noqa: E402

BF16 = torch.bfloat16


class Model:
    """Embedding, bias and head, their fp32 masters, optimizer states and gradients."""

    def __init__(self, vocab: int, width: int, seed: int):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.master = {"embed": torch.randn(vocab, width, generator=g, device="cuda") * 0.3,
                       "bias": torch.zeros(width, device="cuda"),
                       "head": torch.randn(vocab, width, generator=g, device="cuda") * 0.05}
        self.param = {k: v.to(BF16) for k, v in self.master.items()}
        self.grad = {k: torch.zeros_like(v) for k, v in self.param.items()}
        views = []
        for name, master in self.master.items():
            small = name != "bias"                       # matrices: 8-bit states, no decay on the bias
            state = lambda: torch.zeros_like(master, dtype=torch.uint8 if small else torch.float32)
            blocks = -(-master.numel() // zs.ZS_ADAM8_BLOCK)
            scale = lambda: torch.zeros(blocks, device="cuda") if small else None
            views.append(zs.TensorView(self.grad[name], master, state(), state(), param=self.param[name],
                                       m_scale=scale(), v_scale=scale(), decay_mult=1.0 if small else 0.0))
        self.tensors = zs.TensorList(views)

    def forward(self, tokens: torch.Tensor):
        x = (self.param["embed"][tokens] + self.param["bias"]).float()
        h = torch.nn.functional.gelu(x).to(BF16)
        return h @ self.param["head"].t(), x, h

    def backward(self, tokens, x, h, dlogits):
        self.grad["head"].copy_(dlogits.t() @ h)
        t = x * 0.7071067811865476
        slope = 0.5 * (1.0 + torch.erf(t)) + x * 0.3989422804014327 * torch.exp(-t * t)
        dx = (dlogits @ self.param["head"]).float() * slope
        self.grad["bias"].copy_(dx.sum(0))
        self.grad["embed"].zero_().index_add_(0, tokens, dx.to(BF16))


class TiedModel:
    """One matrix for embedding and head, and a norm between; fp32 masters, bf16 copy of the matrix."""

    def __init__(self, vocab: int, width: int, tokens: int, seed: int):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        new = lambda *n, dtype=torch.float32: torch.empty(*n, dtype=dtype, device="cuda")
        self.master = {"table": torch.randn(vocab, width, generator=g, device="cuda") * width ** -0.5,
                       "gamma": torch.ones(width, device="cuda"), "beta": torch.zeros(width, device="cuda")}
        self.table = self.master["table"].to(BF16)
        self.grad = {"table": new(vocab, width, dtype=BF16), "gamma": new(width), "beta": new(width)}
        self.scale = width ** 0.5
        self.x, self.y, self.dy, self.dx = (new(tokens, width, dtype=BF16) for _ in range(4))
        self.stats, self.saved, self.logp = new(tokens, 2), new(tokens, 2), new(tokens)
        self.head_work, self.norm_work = zs.new_head_work(tokens, width, vocab), zs.new_layer_norm_work(tokens, width)
        self.embed_work = zs.new_embed_work(tokens, width)
        self.tensors = zs.TensorList([
            zs.TensorView(self.grad[k], m, torch.zeros_like(m), torch.zeros_like(m), param=self.table if k == "table" else None,
                          decay_mult=1.0 if k == "table" else 0.0) for k, m in self.master.items()])

    def gradients(self, tokens, label, dlogp, ctrl):
        """Log-probabilities of the labels, and the loss-scaled gradient of sum dlogp logp."""
        m = self.master
        zs.zero_embed_async(self.table, tokens, self.x, scale=self.scale)
        zs.zero_layer_norm_async(self.x, m["gamma"], m["beta"], self.y, saved=self.stats)
        zs.zero_head_logp_async(self.y, self.table, label, self.logp, self.head_work, saved=self.saved)
        zs.zero_head_logp_grad_async(self.y, self.table, label, self.saved, dlogp, self.dy, self.grad["table"], self.head_work,
                                     ctrl_dev=ctrl)
        zs.zero_layer_norm_grad_async(self.dy, self.x, m["gamma"], self.stats, self.dx, self.grad["gamma"], self.grad["beta"],
                                      self.norm_work)
        zs.zero_embed_grad_async(tokens, self.dx, self.grad["table"], self.embed_work, scale=self.scale, accumulate=True)


def run_supervised(steps: int = 30, vocab: int = 5003, width: int = 256, tokens: int = 768, seed: int = 0):
    """Trains the tied model on next tokens for `steps` steps; returns each step's mean
    log-probability of the labels, and the control block."""
    model = TiedModel(vocab, width, tokens, seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1)
    last, label = (torch.randint(0, vocab, (tokens,), generator=g, device="cuda") for _ in range(2))
    label[torch.arange(tokens, device="cuda") % 12 < 4] = -100      # of each sequence of 12: four tokens of prompt
    live = (label >= 0).float()
    dlogp = -live / live.sum()                                      # the mean cross entropy's
    ctrl, work, sqnorm, adam = zs.new_ctrl(), zs.new_work(), zs.new_sqnorm(), zs.adam(3e-3, 0.9, 0.95, 1e-8, 0.01)
    zs.zero_ctrl_init(ctrl, 256.0)
    history = []
    for _ in range(steps):
        model.gradients(last, label, dlogp, ctrl)
        zs.zero_tensors_sqnorm_async(model.tensors, sqnorm, work, ctrl)
        zs.zero_tensors_adamw_async(model.tensors, adam, ctrl, max_norm=1.0, sqnorm_dev=sqnorm)
        history.append(-(model.logp * dlogp).sum())
    return torch.stack(history).cpu(), zs.read_ctrl(ctrl)


def run(loss: str = "policy", steps: int = 30, vocab: int = 5003, width: int = 256, tokens: int = 768, seed: int = 0):
    """Trains for `steps` steps; returns the loss of each."""
    model = Model(vocab, width, seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1)
    draw = lambda *n: torch.randint(0, vocab, n, generator=g, device="cuda")
    new = lambda *n: torch.empty(*n, device="cuda")
    ctrl, work, sqnorm = zs.new_ctrl(), zs.new_work(), zs.new_sqnorm()
    zs.zero_ctrl_init(ctrl, 256.0)
    adam = zs.adam(3e-3, 0.9, 0.95, 1e-8, 0.01)
    last, label = draw(tokens), draw(tokens)
    prompt = torch.arange(tokens, device="cuda") % 12 < 4           # of each sequence of 12: four tokens of prompt
    label[prompt] = -100
    logp, entropy, saved = new(tokens), new(tokens), new(tokens, 2)
    logits, _, _ = model.forward(last)
    zs.zero_token_logp_async(logits, label, logp, entropy=entropy, saved=saved)
    ref = logp.clone()
    history = []
    if loss == "policy":
        # a token is good if its number is even
        advantage = torch.where(label % 2 == 0, 1.0, -1.0)
        weights = (~prompt).float() / (~prompt).sum()
        hp, totals = zs.policy(0.2, 0.28, 3.0, kl_coef=0.02, entropy_coef=1e-3), new(zs.ZS_POLICY_TOTALS)
    else:
        # sequences of 12 tokens in turn chosen and rejected
        cu = torch.arange(0, tokens + 1, 12, device="cuda")
        pairs = (len(cu) - 1) // 2
        hp, totals = zs.preference(0.1, "sigmoid"), new(zs.ZS_PREFERENCE_TOTALS)
        pair_loss, reward, dlogp = new(pairs), new(2 * pairs), new(tokens)
    old = logp.clone()
    for step in range(steps):
        logits, x, h = model.forward(last)
        if loss == "policy":
            if step % 4 == 0:                                       # sample anew: here, the same tokens' new scores
                zs.zero_token_logp_async(logits, label, old)
            zs.zero_policy_loss_async(logits, label, old, advantage, weights, hp, totals, work, ref_logp=ref,
                                      logp=logp, dlogits=logits, ctrl_dev=ctrl)
        else:
            zs.zero_token_logp_async(logits, label, logp, saved=saved)
            zs.zero_preference_loss_async(logp, cu, hp, pair_loss, reward, totals, work, ref_logp=ref, mask=~prompt,
                                          dlogp=dlogp)
            zs.zero_token_logp_grad_async(logits, label, saved, dlogp, logits, ctrl_dev=ctrl)
        model.backward(last, x, h, logits)                          # the logits are their gradient by now
        zs.zero_tensors_sqnorm_async(model.tensors, sqnorm, work, ctrl)
        zs.zero_tensors_adamw_async(model.tensors, adam, ctrl, max_norm=1.0, sqnorm_dev=sqnorm)
        history.append(totals.clone())
    return torch.stack(history).cpu(), logp.cpu(), ref.cpu(), label.cpu(), zs.read_ctrl(ctrl)


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=30)
    ap.add_argument("--loss", choices=("policy", "preference", "supervised"), default="policy")
    a = ap.parse_args()
    if a.loss == "supervised":
        mean, ctrl = run_supervised(a.steps)
        for i in range(0, a.steps, max(1, a.steps // 10)):
            print(f"step {i:3d}  mean log-probability {mean[i]:9.5f}")
        print(f"{ctrl['step']} steps, {ctrl['skipped']} skipped")
        return
    totals, logp, ref, label, ctrl = run(a.loss, a.steps)
    for i in range(0, a.steps, max(1, a.steps // 10)):
        print(f"step {i:3d}  totals " + "  ".join(f"{x:9.5f}" for x in totals[i].tolist()))
    good = (label >= 0) & (label % 2 == 0)
    print(f"mean log-probability of even tokens {ref[good].mean():.3f} -> {logp[good].mean():.3f}; "
          f"{ctrl['step']} steps, {ctrl['skipped']} skipped")


if __name__ == "__main__":
    main()
