"""What the cross entropy's contract says of rows without a probability, of zero rows beside infinite weights, and of
weights of very different sizes."""
import pytest
import torch

from tests import block_oracle as o
from tests.block_oracle import BF16, F16, F32
from tests.test_gpu_entropy import Case

pytestmark = pytest.mark.gpu

# T, V, K: split, pairs whose logits are multiplied again, pairs with kept exponentials
SIZES = [(40, 300, 64), (600, 700, 64), (600, 700, 512)]


@pytest.mark.parametrize("T,V,K", SIZES)
def test_rows_of_nothing_but_minus_infinity(T, V, K):
    """lse is -inf, the loss and the gradients are NaN; other tokens' dX is theirs."""
    c = Case(T, V, K, BF16, gdt=F32)
    c.x[:] = 0
    c.x[:, 0] = 1
    c.x[5, 0], c.x[5, 1] = 0, 1
    c.w[:, 1] = -3.0e38
    c.x[5, 2], c.w[:, 2] = 1, -3.0e38        # two of the largest numbers: a float32 sum of -inf, W finite
    c.w[:, 0] = torch.randn((V,), generator=torch.Generator().manual_seed(3)).cuda()
    c.call()
    bad = torch.zeros((T,), dtype=torch.bool, device="cuda")
    bad[5] = True
    assert c.lse[5] == -float("inf") and c.lse[~bad].isfinite().all()
    assert torch.equal(c.loss.isnan(), bad) and c.stats[0].isnan()
    assert torch.equal(c.dx.isnan().any(1), bad) and c.dx[5].isnan().all()
    assert c.dw[:, 1].isnan().all()
