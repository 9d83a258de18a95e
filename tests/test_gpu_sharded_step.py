"""The sharded training step (examples/sharded_policy_step.py) end to end: its first step against
autograd in float64 on the same 16-bit weights, and that training does what the loss says."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location(
        "sharded_policy_step", os.path.join(ROOT, "examples", "sharded_policy_step.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_first_step_against_autograd():
    ex = example()
    model = ex.ShardedModel(W=2, tokens=64, dim=72, hidden=96, vocab=200, state_bits=32, seed=3)
    batch = ex.make_batch(model, seed=4)
    noise = torch.randn(batch["old"].shape, generator=torch.Generator().manual_seed(5)).cuda()
    batch["old"] = batch["old"] + 0.3 * noise
    batch["ref"] = batch["ref"] - 0.2 * noise
    w1, w2 = (model.master[n].to(torch.bfloat16).double().requires_grad_(True) for n in ("w1", "w2"))
    b1 = model.master["b1"].double().requires_grad_(True)
    before = {n: m.clone() for n, m in model.master.items()}
    stats, logp = model.step(batch, lr=1e-3, kl_coef=0.05)
    # the same loss in float64
    x = batch["x"].reshape(-1, model.dim).double()
    h = torch.nn.functional.silu(x @ w1.t() + b1)
    lp = torch.log_softmax(h @ w2.t(), 1).gather(1, batch["target"].reshape(-1, 1))[:, 0]
    old, ref, adv, w = (batch[k].reshape(-1).double() for k in ("old", "ref", "advantage", "weight"))
    r = torch.exp(lp - old)
    loss = (w * (-torch.minimum(r * adv, r.clamp(0.8, 1.2) * adv)
                 + 0.05 * (torch.exp(ref - lp) - (ref - lp) - 1))).sum()
    loss.backward()
    # h, z1, dz1, the logits and their gradient are 16-bit on the way: a few 2^-9 of each other's size
    for name, g in (("w1", w1.grad), ("w2", w2.grad), ("b1", b1.grad)):
        d = (model.grad[name].double() - g).norm() / g.norm()
        assert d <= 8 * 2.0 ** -9, (name, float(d))
    assert abs(float(stats[0]) - float(loss.detach())) <= 2.0 ** -6 * float((w * adv.abs()).sum())
    keep = w > 0
    assert ((logp.reshape(-1).double() - lp)[keep].abs() <= 0.06).all()
    # AdamW's first step moves every parameter against its gradient by lr (1 + eps), after the decay
    for name in ("w1", "w2", "b1"):
        g = model.grad[name].double()
        want = before[name].double() * (1 - 1e-3 * 0.01) - 1e-3 * g / (g.abs() + 1e-8)
        assert ((model.master[name].double() - want).abs() <= 1e-3 * 2.0 ** -14 + 2.0 ** -22 * want.abs()).all()
    for name in ("w1", "w2"):  # the copies that the next gather sends
        rows = model.block_shape(name)[0]
        for q in range(model.W):
            block = model.heap.view(q, model.offsets[name, "block"], *model.block_shape(name), model.shapes[name][1],
                                    torch.bfloat16)
            assert torch.equal(block, model.master[name][q * rows:(q + 1) * rows].to(torch.bfloat16))
    model.gather()
    assert torch.equal(model.whole("w1", 0), model.whole("w1", 1))


@pytest.mark.parametrize("state_bits", [32, 8])
def test_training_raises_what_it_rewards(state_bits):
    ex = example()
    model = ex.ShardedModel(W=4, tokens=256, state_bits=state_bits, seed=1)
    batch = ex.make_batch(model)
    losses = [float(model.step(batch)[0][0]) for _ in range(15)]
    assert losses[-1] < losses[0] - 0.1                       # the ratio of rewarded tokens has grown
    _, logp = model.step(batch)
    gain = (logp - batch["old"]) * (batch["weight"] > 0)
    assert gain[batch["advantage"] > 0].mean() > 0 > gain[batch["advantage"] < 0].mean()
    import gemm_gather_gb300 as gg
    assert gg.device_status() == 0
