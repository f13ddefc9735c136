"""The preference loss at the largest number of pairs that the call takes."""
import math

import pytest
import torch

from test_gpu_losses import U

pytestmark = pytest.mark.gpu


def test_the_largest_number_of_pairs(zs, cuda_device):
    """2^31 - 1 pairs without tokens: the pair that a cluster would take next has
    a number past 31 bits, and sequence numbers need 33.  Each pair's loss is
    ln 2, its weight 2^-31 (the uniform one, rounded to fp32)."""
    pairs = (1 << 31) - 1
    cu = torch.zeros(2 * pairs + 1, dtype=torch.int64, device="cuda")
    loss, reward = torch.full((pairs,), 9.0, device="cuda"), torch.full((2 * pairs,), 9.0, device="cuda")
    totals = torch.full((3,), 9.0, device="cuda")
    zs.zero_preference_loss_async(torch.empty(0, device="cuda"), cu, zs.preference(0.1), loss, reward, totals, zs.new_work())
    del cu
    assert abs(loss[0].item() - math.log(2)) <= 4 * U
    low, high = loss.aminmax()
    assert low.item() == high.item() == loss[0].item()
    low, high = reward.aminmax()
    assert low.item() == high.item() == 0.0
    assert abs(totals[0].item() - math.log(2)) <= 8 * U and totals[1].item() == 0.0 and totals[2].item() == 0.0
