"""The sharded block's training step (examples/sharded_block_step.py) end to end: its gradients against the
formulas in float64 from what the step keeps, and that it runs.

Between the float64 chain and the kernels' lie roundings to bfloat16, half a step of 2^-8 each: of n, z, a, m, h
and y forward (which only the loss sees; the backward pass starts from what was kept), of the logits' gradient,
dy, dh, dz and dn backward.  A gradient is behind at most four of the latter, each relative to its own size
and of either sign: 4 x 2^-8 of its norm.
"""
import importlib.util
import os

import pytest
import torch

from tests import block_oracle as o

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("sharded_block_step", os.path.join(ROOT, "examples", "sharded_block_step.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def norm_gradient(h, rstd, w, dy, along=None):
    u, g = h * rstd[:, None], dy * w
    dh = rstd[:, None] * (g - u * (g * u).mean(1, keepdim=True))
    return dh if along is None else dh + along, (dy * u).sum(0)


def test_gradients_of_a_step():
    ex = example()
    model = ex.ShardedBlock(W=2, tokens=96, dim=144, hidden=272, vocab=1002, seed=3)
    batch = ex.make_batch(model, seed=4)
    masked = batch["weight"] == 0
    batch["target"][masked] = -5
    model.gather()
    w = {n: model.whole(n, 0).double() for n in model.shapes}
    g1, g2 = (model.master[g].double().clone() for g in ("g1", "g2"))
    want = {n: torch.zeros_like(m, dtype=torch.float64) for n, m in model.master.items()}
    loss, dx = 0.0, []
    for r in range(model.W):
        x, tw = batch["x"][r].double(), batch["weight"][r].double()
        tg = torch.where(masked[r], 0, batch["target"][r])
        y, k = model.forward(batch["x"][r], r)
        n, z = o.values(k["nc"].view(torch.float8_e4m3fn), k["ns"]), o.values(k["zc"].view(torch.float8_e4m3fn), k["zs"])
        # what was kept is what the forward pass computed: 8 bits of the norm and of its product
        rstd = 1 / torch.sqrt(x.square().mean(1) + ex.EPS)
        n64 = x * rstd[:, None] * g1
        assert ((n - n64).norm() <= 2.0 ** -4 * n64.norm()) and ((z - n64 @ w["w1"].t()).norm() <= 2.0 ** -4 * z.norm())
        h, y64 = k["h"].double(), y.double()
        logits = y64 @ w["wv"].t()
        lse = torch.logsumexp(logits, 1)
        loss += float((tw * (lse - logits.gather(1, tg[:, None])[:, 0])).sum())
        dl = tw[:, None] * (torch.softmax(logits, 1) - torch.nn.functional.one_hot(tg, model.vocab).double())
        want["wv"] += dl.t() @ y64
        dh, d = norm_gradient(h, k["rstd2"].double(), g2, dl @ w["wv"])
        want["g2"] += d
        a, slope = o.act64(z, "silu"), o.slope64(z, "silu")
        want["w2"] += dh.t() @ a
        dz = (dh @ w["w2"]) * slope
        want["w1"] += dz.t() @ n
        d, dg = norm_gradient(x, k["rstd1"].double(), g1, dz @ w["w1"], dh)
        want["g1"] += dg
        dx.append(d)
    before = {n: m.clone() for n, m in model.master.items()}
    stats, losses, got = model.step(batch)
    assert abs(float(stats[0]) - loss) <= 1e-5 * loss and abs(float(stats[1]) - 1) < 1e-6
    assert (losses[masked] == 0).all()
    for name in want:
        d = (model.grad[name].double() - want[name]).norm() / want[name].norm()
        assert d <= 4 * 2.0 ** -8, (name, float(d))
    dx = torch.stack(dx)
    assert (got.double() - dx).norm() <= 4 * 2.0 ** -8 * dx.norm()
    assert (got[masked] == 0).all()
    for name in model.master:       # AdamW's first step moves every parameter that has a gradient
        moved = (model.master[name] != before[name]) | (model.grad[name] == 0)
        assert moved.all(), name
    for name in model.shapes:       # the copies that the next gather sends
        rows = model.shapes[name][0] // model.W
        for q in range(model.W):
            block = model.heap.view(q, model.offsets[name, "block"], rows, model.shapes[name][1], model.shapes[name][1],
                                    torch.bfloat16)
            assert torch.equal(block, model.master[name][q * rows:(q + 1) * rows].to(torch.bfloat16))


def test_steps_in_a_graph_and_twice():
    """A captured step gives the eager step's gradients, bit by bit, and so does the same step again."""
    import gemm_gather_gb300 as gg
    ex = example()
    results = []
    for how in ("eager", "eager", "graph"):
        model = ex.ShardedBlock(W=2, tokens=256, seed=5)
        batch = ex.make_batch(model, seed=6)
        model.gather()

        def passes():
            for r in range(model.W):
                b = {k: v[r] for k, v in batch.items()}
                y, kept = model.forward(b["x"], r)
                model.backward(b["x"], y, kept, b, r, accumulate=r > 0)
        if how == "graph":
            passes()
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                passes()
            for g in model.grad.values():
                g.zero_()
            graph.replay()
        else:
            passes()
        torch.cuda.synchronize()
        results.append({n: g.clone() for n, g in model.grad.items()})
    for other in results[1:]:
        for n, g in results[0].items():
            assert torch.equal(g, other[n]), n
    assert gg.device_status() == 0


def test_the_example_runs(capsys):
    ex = example()
    model = ex.ShardedBlock(W=4, tokens=256)
    batch = ex.make_batch(model)
    for _ in range(3):
        stats, _, _ = model.step(batch)
    assert torch.isfinite(stats).all()
