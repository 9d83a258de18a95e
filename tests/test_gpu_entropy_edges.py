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


@pytest.mark.parametrize("T,V,K", SIZES)
@pytest.mark.parametrize("layout", ["nk", "kn"])
def test_rows_that_fill_up_a_block_stay_zero_whatever_the_weights_hold(T, V, K, layout):
    """Tokens that count are padded to 64 with rows of zeros, whose logits beside infinite weights are NaN: dW meets
    nothing of them."""
    weights = torch.zeros((T,))
    weights[: T - 23 - T % 64] = 1.0 / T
    assert int((weights != 0).sum()) % 64 != 0
    c = Case(T, V, K, BF16, layout, weights=weights, gdt=F32, dx=False)
    c.x[:] = c.x.abs() + 0.1
    rows = c.w if layout == "nk" else c.w.t()
    rows[3], rows[V - 1] = -float("inf"), -float("inf")
    c.target[(c.target == 3) | (c.target == V - 1)] = 7
    c.call()
    got = c.dw if layout == "nk" else c.dw.t()
    assert got.isfinite().all() and (got[3] == 0).all() and (got[V - 1] == 0).all()
    # the others' are what they are without the two
    d = Case(T, V, K, BF16, layout, weights=weights, gdt=F32, dx=False)
    d.x.copy_(c.x), d.w.copy_(c.w), d.target.copy_(c.target)
    rows = d.w if layout == "nk" else d.w.t()
    rows[3], rows[V - 1] = -1e4, -1e4
    d.call()
    assert torch.equal(got, d.dw if layout == "nk" else d.dw.t())


@pytest.mark.parametrize("T,V,K", SIZES)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_weights_of_very_different_sizes(T, V, K, dtype):
    """2^0 to 2^-20 of the largest.  In bfloat16 every dX row is as near as its own weight's; in float16 terms of a
    gradient below 2^-38 of the largest weight are lost, which check() allows for."""
    weights = torch.exp2(-torch.randint(0, 21, (T,), generator=torch.Generator().manual_seed(T)).float())
    weights[0] = 1.0
    c = Case(T, V, K, dtype, weights=weights, gdt=F32)
    c.call(grad_scale=1024.0).check(grad_scale=1024.0)


@pytest.mark.parametrize("T,V,K", SIZES)
def test_float16_keeps_its_precision_down_to_its_limit(T, V, K):
    """A token of weight r times the largest: probabilities from 2^-27 / r on keep half a step of 2^-11, and that
    of a kept exponential.  Flat softmax over V <= 700 entries (p above 2^-10.5), r = 2^-16."""
    weights = torch.full((T,), 2.0 ** -16)
    weights[1] = 1.0
    c = Case(T, V, K, F16, weights=weights, scale=0.05, dw=False)
    scale = 2.0 ** 16
    c.call(grad_scale=scale)
    x, w = c.x.double(), c.w.double()
    z = x @ w.t()
    p = torch.softmax(z, 1)
    assert float(p.min()) >= 2.0 ** -11
    dz = c.weight.double()[:, None] * scale * (p - torch.zeros_like(p).scatter_(1, c.target[:, None], 1.0))
    # what a logit is off by (test_gpu_entropy.py), once in a probability and once in the sum
    e = (x.abs() @ w.abs().t()) * (K * 2.0 ** -23)
    err = dz.abs() * (2.0 ** -11 + 2.0 ** -12) + c.weight.double()[:, None] * scale * p * (2 * e + 2.0 ** -19)
    bound = err @ w.abs() + (dz.abs() @ w.abs()) * (V * 2.0 ** -23)
    want = dz @ w
    small = torch.arange(T, device="cuda") != 1
    assert ((c.dx.double() - want).abs() <= bound + o.half_ulp(want, F16) * 1.01)[small].all()
