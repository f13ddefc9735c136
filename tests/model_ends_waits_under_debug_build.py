"""Run under the debug build by test_gpu_model_ends_waits.py: the head's products with
waits that give up after a few tries, or at once."""
import pytest
import torch

from test_gpu_head import _inputs

pytestmark = pytest.mark.gpu

DEFAULT = 1 << 20


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,vocab,width", [(3, 5000, 512), (100, 3000, 1600), (300, 40_000, 256), (1500, 9000, 768)])
def test_a_wait_that_runs_out_shows_as_nan(zs, cuda_device, rows, vocab, width, dtype):
    h, w, y, g = _inputs(rows, vocab, width, dtype, rows + vocab)
    y[::4] = -1
    live = y >= 0
    work, wide = zs.new_head_work(rows, width, vocab), 8
    saved0, logp0 = torch.empty(rows, 2, device="cuda"), torch.empty(rows, device="cuda")
    zs.zero_head_logp_async(h, w, y, logp0, work, saved=saved0)
    dlogp = torch.rand(rows, generator=g, device="cuda") + 0.5

    def call():
        logp = torch.full((rows + 2 * wide,), 7.0, device="cuda")
        dh, dw = (torch.full((n, width + 2 * wide), 7.0, dtype=dtype, device="cuda") for n in (rows, vocab))
        zs.zero_head_logp_async(h, w, y, logp[wide:-wide], work)
        zs.zero_head_logp_grad_async(h, w, y, saved0, dlogp, dh[:, wide:-wide], dw[:, wide:-wide], work)
        torch.cuda.synchronize()
        for t in (dh, dw):
            assert (t[:, :wide] == 7).all() and (t[:, -wide:] == 7).all()
        assert (logp[:wide] == 7).all() and (logp[-wide:] == 7).all()
        return [t.float() for t in (logp[wide:-wide], dh[:, wide:-wide], dw[:, wide:-wide])]

    want = call()
    assert all(t.isfinite().all() for t in want) and torch.equal(want[0], logp0)
    try:
        for tries in (0, 1, 2, 4, 16):
            assert zs.lib().zero_debug_wait_limit(tries) == 1
            got = call()
            for a, b in zip(got, want):
                assert (a.isnan() | (a == b)).all(), tries
            if tries == 0:
                assert got[0][live].isnan().all() and got[1][live].isnan().all() and got[2].isnan().all()
                assert (got[0][~live] == 0).all() and (got[1][~live] == 0).all()
    finally:
        assert zs.lib().zero_debug_wait_limit(DEFAULT) == 1
    again = call()
    assert all(torch.equal(a, b) for a, b in zip(again, want))
