"""Training steps of a two-layer model whose weights are held as row blocks by the ranks of a heap.

    logits = silu(x W1^T + b1) W2^T

Every logical rank owns a row block of W1 and of W2 (a float32 master, its AdamW state, and the 16-bit
copy in its heap partition) and a shard of the tokens.  One step is

    all_gather        the 16-bit row blocks become the whole weights, in every partition
    linear            each rank's tokens through its partition's weights, Z of layer 1 kept
    policy_loss       the clipped loss with a KL term; the logits become their own gradient in place
    linear_backward   layer 2: dZ1 = (dlogits W2) silu'(Z1) and dW2; layer 1: dW1 and db1, float32,
                      accumulated over the ranks' tokens
    adamw             every row block's master, its states, and the 16-bit copy for the next gather

Run:  python examples/sharded_policy_step.py [--steps 20] [--state-bits 8]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import gemm_gather_gb300 as gg  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32


class ShardedModel:
    """Weights W1 (hidden x dim) and W2 (vocab x hidden) as row blocks of W ranks, tokens as shards."""

    def __init__(self, W=4, tokens=512, dim=256, hidden=512, vocab=1024, state_bits=32, seed=0):
        assert hidden % W == 0 and vocab % W == 0 and tokens % W == 0
        self.W, self.T, self.dim, self.hidden, self.vocab = W, tokens // W, dim, hidden, vocab
        self.state_bits = state_bits
        self.programs = torch.cuda.get_device_properties(0).multi_processor_count
        # a partition: the rank's own row blocks, then the gathered weights
        self.shapes = {"w1": (hidden, dim), "w2": (vocab, hidden)}
        self.offsets, at = {}, 0
        for name, (rows, cols) in self.shapes.items():
            for part, r in (("block", rows // W), ("whole", rows)):
                self.offsets[name, part] = at
                at += (r * cols * 2 + 255) // 256 * 256
        self.heap = gg.SymmetricHeap(W, at, device="cuda")
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        self.master = {n: torch.randn(s, generator=gen, device="cuda") * s[1] ** -0.5 for n, s in self.shapes.items()}
        self.master["b1"] = torch.zeros((hidden,), device="cuda")
        self.grad = {n: torch.zeros_like(m) for n, m in self.master.items()}
        tensors = []
        for name in self.shapes:
            for r in range(W):
                block = self.heap.view(r, self.offsets[name, "block"], *self.block_shape(name), self.shapes[name][1], BF16)
                rows = slice(r * block.shape[0], (r + 1) * block.shape[0])
                block.copy_(self.master[name][rows])
                tensors.append(self._optimized(self.master[name][rows], self.grad[name][rows], block))
        tensors.append(self._optimized(self.master["b1"], self.grad["b1"], None))
        self.tensors = tensors
        self.table = gg.adamw_tensors(tensors, state_bits=state_bits)
        self.step_count = 0

    def block_shape(self, name):
        rows, cols = self.shapes[name]
        return rows // self.W, cols

    def _optimized(self, param, grad, copy):
        n, dt = param.numel(), torch.float8_e4m3fn if self.state_bits == 8 else F32
        t = {"param": param, "grad": grad, "m": torch.zeros((n,), dtype=dt, device="cuda"),
             "v": torch.zeros((n,), dtype=dt, device="cuda"), "copy": copy}
        if self.state_bits == 8:
            blocks = -(-n // gg.ADAMW_BLOCK)
            t["m_scale"], t["v_scale"] = (torch.ones((blocks,), device="cuda") for _ in range(2))
        return t

    def whole(self, name, r):
        rows, cols = self.shapes[name]
        return self.heap.view(r, self.offsets[name, "whole"], rows, cols, cols, BF16)

    def gather(self):
        for name in self.shapes:
            rows, cols = self.block_shape(name)
            gg.all_gather(self.heap.heap, -1, self.heap.ptr(0, self.offsets[name, "block"]), cols,
                          self.heap.ptr(0, self.offsets[name, "whole"]), cols, rows, cols, BF16, (8, 256),
                          self.programs, (0, 1, self.W))

    def forward(self, x, r):
        """Logits of rank r's tokens, and what the backward pass needs."""
        z1, h = (torch.empty((self.T, self.hidden), dtype=BF16, device="cuda") for _ in range(2))
        logits = torch.empty((self.T, self.vocab), dtype=BF16, device="cuda")
        gg.linear(x, self.dim, self.whole("w1", r), self.dim, "nk", self.master["b1"], "silu", None, 0, h, self.hidden,
                  z1, self.hidden, self.T, self.hidden, self.dim, BF16)
        gg.linear(h, self.hidden, self.whole("w2", r), self.hidden, "nk", None, "none", None, 0, logits, self.vocab,
                  None, 0, self.T, self.vocab, self.hidden, BF16)
        return logits, h, z1

    def backward(self, x, dlogits, h, z1, r, accumulate):
        dz1 = torch.empty_like(z1)
        gg.linear_backward(dlogits, self.vocab, h, self.hidden, self.whole("w2", r), self.hidden, "nk", z1, self.hidden,
                           "silu", dz1, self.hidden, self.grad["w2"], self.hidden, None, F32, accumulate, self.T,
                           self.vocab, self.hidden, BF16)
        gg.linear_backward(dz1, self.hidden, x, self.dim, None, self.dim, "nk", None, 0, "none", None, 0,
                           self.grad["w1"], self.dim, self.grad["b1"], F32, accumulate, self.T, self.hidden, self.dim, BF16)

    def step(self, batch, lr=1e-3, kl_coef=0.02):
        """One step; the statistics of the loss (loss, KL, clipped share, ratio) and every token's log probability."""
        self.gather()
        stats = torch.empty((self.W, 4), device="cuda")
        logp = torch.empty((self.W, self.T), device="cuda")
        for r in range(self.W):
            b = {k: v[r] for k, v in batch.items()}
            logits, h, z1 = self.forward(b["x"], r)
            gg.policy_loss(logits, self.vocab, b["target"], b["old"], b["ref"], b["advantage"], b["weight"], self.T,
                           self.vocab, BF16, stats[r], logp[r], logits, self.vocab, kl_coef=kl_coef)
            self.backward(b["x"], logits, h, z1, r, accumulate=r > 0)
        self.step_count += 1
        gg.adamw(self.table, self.step_count, lr, seed=self.step_count)
        return stats.sum(0), logp


def make_batch(model, seed=1, masked=0.25):
    """Tokens of W shards: targets to be made likelier or less likely, some of them masked; the old and the
    reference policy are the model's own first log probabilities."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    W, T = model.W, model.T
    b = {"x": torch.randn((W, T, model.dim), generator=gen, device="cuda").to(BF16),
         "target": torch.randint(0, model.vocab, (W, T), generator=gen, device="cuda"),
         "advantage": torch.where(torch.rand((W, T), generator=gen, device="cuda") < 0.8, 1.0, -0.5)}
    keep = torch.rand((W, T), generator=gen, device="cuda") >= masked
    b["weight"] = keep.float() / keep.sum()
    model.gather()
    first = torch.empty((W, T), device="cuda")
    for r in range(W):
        logits, _, _ = model.forward(b["x"][r], r)
        gg.policy_loss(logits, model.vocab, b["target"][r], None, None, b["advantage"][r], torch.ones_like(first[r]), T,
                       model.vocab, BF16, None, first[r], None, 0)
    b["old"], b["ref"] = first.clone(), first.clone()
    return b


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--state-bits", type=int, default=8, choices=(8, 32))
    ap.add_argument("--ranks", type=int, default=4)
    args = ap.parse_args()
    model = ShardedModel(W=args.ranks, state_bits=args.state_bits)
    batch = make_batch(model)
    for k in range(args.steps):
        stats, _ = model.step(batch)
        loss, kl, clipped, ratio = stats.tolist()
        print(f"step {k + 1:3d}  loss {loss:+.4f}  kl {kl:.4f}  clipped {clipped:.2f}  ratio {ratio:.3f}")


if __name__ == "__main__":
    main()
