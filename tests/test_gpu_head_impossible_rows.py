"""The head's gradient next to a row whose logits are all -inf: such a row has no
gradient, so the call's outputs are those of the same call with that row's label ignored."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows", [1, 6, 128, 700, 1024, 1025, 9000])
def test_row_of_nothing_but_minus_infinity(zs, cuda_device, rows, dtype):
    vocab, width = 600, 64
    g = torch.Generator(device="cuda")
    g.manual_seed(rows)
    h = torch.randn(rows, width, generator=g, device="cuda").to(dtype)
    w = (torch.randn(vocab, width, generator=g, device="cuda") * 0.3).to(dtype)
    w[:, 5] = 0.25
    y = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    none = torch.arange(rows, device="cuda") % 5 == 0
    h[none] = 0.0
    h[none, 5] = -math.inf                                   # against positive weights
    work = zs.new_head_work(rows, width, vocab)
    logp, saved = torch.empty(rows, device="cuda"), torch.empty(rows, 2, device="cuda")
    zs.zero_head_logp_async(h, w, y, logp, work, saved=saved)
    assert (logp[none] == -math.inf).all() and (saved[none, 1] == -math.inf).all() and logp[~none].isfinite().all()
    dlogp = torch.randn(rows, generator=g, device="cuda")
    got, want = [], []
    for labels, out in ((y, got), (torch.where(none, -100, y), want)):
        dh, dw = torch.full_like(h, 7.0), torch.full_like(w, 7.0)
        zs.zero_head_logp_grad_async(h, w, labels, saved, dlogp, dh, dw, work)
        out += [dh, dw]
    assert (got[0][none] == 0).all() and got[1].isfinite().all()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
