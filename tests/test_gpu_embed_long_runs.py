"""The embedding's gradient where one id fills thousands of chunks of the sorted list: small
integers, so that every order of a sum gives the same result."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [(1 << 16) + 1, (1 << 20) + 5, 1 << 21])
@pytest.mark.parametrize("width", [1, 8])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_runs_of_thousands_of_chunks(zs, cuda_device, n, width, dtype):
    vocab = 9
    dout = ((torch.arange(n, device="cuda")[:, None] * 7 + torch.arange(width, device="cuda")[None]) % 5 - 2).to(dtype)
    work = zs.new_embed_work(n, width)
    start = torch.arange(vocab * width, device="cuda").view(vocab, width).float()
    cuts = [(), (n // 2,), (1, n - 1), (64, 64 * 33), (64 * 31 + 7, 64 * 1024 + 7, 64 * 1025 + 8), (n // 3, n // 3 + 64 * 32)]
    for cut in cuts:
        ids = sum(((torch.arange(n, device="cuda") >= c).long() for c in cut), torch.zeros(n, dtype=torch.int64, device="cuda"))
        shuffled = torch.randperm(n, device="cuda")
        want = torch.zeros(vocab, width, dtype=torch.float64, device="cuda").index_add_(0, ids, dout[shuffled.argsort()].double())
        for add in (False, True):
            table = start.clone()
            zs.zero_embed_grad_async(ids[shuffled], dout, table, work, accumulate=add)
            assert torch.equal(table.double(), want + start.double() if add else want)
