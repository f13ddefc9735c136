"""Run under the debug build by test_gpu_waits.py: the logits kernels with waits
that give up after a few tries, or at once."""
import pytest
import torch

from test_gpu_losses import _policy_inputs

pytestmark = pytest.mark.gpu

DEFAULT = 1 << 20
# rows, vocabulary: clusters of eight, of four and of one; rows in several turns
SHAPES = [(3, 200_003), (24, 50_257), (3000, 1500), (700, 32_000), (64, 131_072)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,vocab", SHAPES)
@pytest.mark.parametrize("op", ["logp", "logp_grad", "policy_loss", "policy"])
def test_a_wait_that_runs_out_shows_as_nan(zs, cuda_device, op, rows, vocab, dtype):
    x, y, old, ref, adv, g = _policy_inputs(rows, vocab, dtype, rows + vocab)
    w = (torch.rand(rows, generator=g, device="cuda") + 0.5) / rows
    if rows > 3:
        w[torch.rand(rows, generator=g, device="cuda") < 0.3] = 0.0
        y[w == 0] = -1
    live = w != 0
    hp, work, wide = zs.policy(dual_clip=2.0, kl_coef=0.1, entropy_coef=0.01), zs.new_work(), 5
    saved, ent0, lp0 = (torch.empty(k, device="cuda") for k in (2 * rows, rows, rows))
    zs.zero_token_logp_async(x, y, lp0, entropy=ent0, saved=saved)

    def call():
        """Every row's outputs side by side, the totals, and the canaries."""
        f = lambda k: torch.full((k + 2 * wide,), 7.0, device="cuda")
        o = {k: f(n) for k, n in (("logp", rows), ("entropy", rows), ("saved", 2 * rows), ("loss", rows), ("totals", 5))}
        v = {k: t[wide:-wide] for k, t in o.items()}
        big = torch.full((rows, vocab + 2 * wide), 7.0, dtype=dtype, device="cuda")
        d = big[:, wide:wide + vocab]
        parts, totals = [], None
        if op == "logp":
            zs.zero_token_logp_async(x, y, v["logp"], entropy=v["entropy"], saved=v["saved"])
            parts = [v["logp"], v["entropy"], v["saved"]]
        elif op == "logp_grad":
            zs.zero_token_logp_grad_async(x, y, saved, adv, d, entropy=ent0, dentropy=old)
            parts = [d]
        else:
            zs.zero_policy_loss_async(x, y, old, adv, w, hp, v["totals"], work, ref_logp=ref, logp=v["logp"], entropy=v["entropy"],
                                      token_loss=v["loss"], dlogits=d if op == "policy" else None)
            parts, totals = [v["logp"], v["entropy"], v["loss"]] + ([d] if op == "policy" else []), v["totals"]
        torch.cuda.synchronize()
        for t in o.values():
            assert (t[:wide] == 7).all() and (t[-wide:] == 7).all()
        assert (big[:, :wide] == 7).all() and (big[:, wide + vocab:] == 7).all()
        return torch.cat([p.reshape(rows, -1).float() for p in parts], 1), totals

    want, want_totals = call()
    assert want.isfinite().all()
    gave_up = 0
    try:
        for tries in (0, 1, 2, 4, 16):
            assert zs.lib().zero_debug_wait_limit(tries) == 1
            got, totals = call()
            nan, same = got.isnan().all(1), (got == want).all(1)
            assert (nan | same).all(), (tries, torch.nonzero(~(nan | same))[:5])
            gave_up += int(nan.sum())
            if tries == 0:
                assert nan[live].all()
            if totals is not None:
                assert torch.equal(totals, want_totals) if not nan.any() else totals.isnan().all()
    finally:
        assert zs.lib().zero_debug_wait_limit(DEFAULT) == 1
    assert gave_up >= int(live.sum())
    again, totals = call()
    assert torch.equal(again, want) and (totals is None or torch.equal(totals, want_totals))
