"""The bound on the vocabulary's losses sees what it is meant to see: logits in 16 bits fail it, float32
logits pass it, at every length that it is used at."""
import pytest
import torch

from tests import entropy_oracle as e


@pytest.mark.parametrize("K,chunk", [(520, 520), (1000, 1000), (1792, 1792), (2100, 1024), (3584, 1024)])
def test_losses_of_rounded_logits_fail(K, chunk):
    g = torch.Generator().manual_seed(K)
    T, V = 120, 1500
    x = torch.randn((T, K), generator=g).to(torch.bfloat16)
    w = (torch.randn((V, K), generator=g) * 2.5 * K ** -0.5).to(torch.bfloat16)
    target = torch.randint(0, V, (T,), generator=g)
    want, lse = e.losses64(x, w, target)
    z = x.float() @ w.float().t()

    def losses(z):
        z = z.double()
        return torch.logsumexp(z, 1) - z.gather(1, target[:, None])[:, 0]
    bound = e.loss_bound(chunk)
    assert e.relative(losses(z), want) < bound / 3
    for t in (torch.float16, torch.bfloat16):
        assert e.relative(losses(z.to(t)), want) > 20 * bound
