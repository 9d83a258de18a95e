"""Training steps of a residual block and a vocabulary head whose memory between the passes is small.

    n = norm(x) g1;  m = silu(n W1^T) W2^T;  y = norm(x + m) g2;  loss = cross entropy of y Wv^T

Every logical rank owns a row block of W1, W2 and Wv (a float32 master, its AdamW state, and the 16-bit
copy in its heap partition) and a shard of the tokens.  One step is

    all_gather            the 16-bit row blocks become the whole weights, in every partition
    rms_norm              n, and n in 8 bits: what the first layer's backward pass needs of it
    linear, pack8         silu(Z) for the second layer, and Z in 8 bits; Z itself is not kept
    rms_norm              the residual's addition and y
    linear_cross_entropy  the loss, dy and dWv, a piece of the vocabulary at a time; no logits
    rms_norm_backward     from dy to the gradient of x + m
    linear_backward8      dW2 and dZ from Z in 8 bits, then dW1 and dn from n in 8 bits
    rms_norm_backward     to x, the gradient along the residual added
    adamw                 every row block's master, its states, and the 16-bit copy for the next gather

Run:  python examples/sharded_block_step.py [--steps 20]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import gemm_gather_gb300 as gg  # noqa: E402

BF16, F32, U8 = torch.bfloat16, torch.float32, torch.uint8
EPS = 1e-6


class ShardedBlock:
    """W1 (hidden x dim), W2 (dim x hidden) and Wv (vocab x dim) as row blocks of W ranks, tokens as shards."""

    def __init__(self, W=4, tokens=512, dim=256, hidden=512, vocab=2048, seed=0):
        assert dim % (8 * W) == 0 and hidden % (8 * W) == 0 and vocab % W == 0 and tokens % W == 0
        self.W, self.T, self.dim, self.hidden, self.vocab = W, tokens // W, dim, hidden, vocab
        self.programs = torch.cuda.get_device_properties(0).multi_processor_count
        self.shapes = {"w1": (hidden, dim), "w2": (dim, hidden), "wv": (vocab, dim)}
        self.offsets, at = {}, 0
        for name, (rows, cols) in self.shapes.items():
            for part, r in (("block", rows // W), ("whole", rows)):
                self.offsets[name, part] = at
                at += (r * cols * 2 + 255) // 256 * 256
        self.heap = gg.SymmetricHeap(W, at, device="cuda")
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        self.master = {n: torch.randn(s, generator=gen, device="cuda") * s[1] ** -0.5 for n, s in self.shapes.items()}
        for g in ("g1", "g2"):
            self.master[g] = torch.ones((dim,), device="cuda")
        self.grad = {n: torch.zeros_like(m) for n, m in self.master.items()}
        tensors = []
        for name, (rows, cols) in self.shapes.items():
            for r in range(W):
                block = self.heap.view(r, self.offsets[name, "block"], rows // W, cols, cols, BF16)
                own = slice(r * block.shape[0], (r + 1) * block.shape[0])
                block.copy_(self.master[name][own])
                tensors.append(self._optimized(self.master[name][own], self.grad[name][own], block))
        tensors += [self._optimized(self.master[g], self.grad[g], None) for g in ("g1", "g2")]
        self.table = gg.adamw_tensors(tensors)
        self.step_count = 0
        # scratch memory of one call at a time, kept for all steps
        T = self.T
        self.scratch = torch.empty((max(gg.linear_cross_entropy_workspace(T, vocab, dim),
                                        gg.linear_backward8_workspace(T, max(dim, hidden)),
                                        gg.rms_norm_backward_workspace(T, dim)),), dtype=U8, device="cuda")

    @staticmethod
    def _optimized(param, grad, copy):
        return {"param": param, "grad": grad, "m": torch.zeros_like(param), "v": torch.zeros_like(param), "copy": copy}

    def whole(self, name, r):
        rows, cols = self.shapes[name]
        return self.heap.view(r, self.offsets[name, "whole"], rows, cols, cols, BF16)

    def gather(self):
        for name, (rows, cols) in self.shapes.items():
            gg.all_gather(self.heap.heap, -1, self.heap.ptr(0, self.offsets[name, "block"]), cols,
                          self.heap.ptr(0, self.offsets[name, "whole"]), cols, rows // self.W, cols, BF16, (8, 256),
                          self.programs, (0, 1, self.W))

    def _room(self, cols, dtype=BF16):
        return torch.empty((self.T, cols), dtype=dtype, device="cuda")

    def _packed(self, cols):
        return self._room(cols, U8), self._room(-(-cols // gg.PACK_BLOCK), F32)

    def forward(self, x, r):
        """y of rank r's tokens, and what the backward pass needs."""
        T, D, H = self.T, self.dim, self.hidden
        n, (nc, ns), rstd1 = self._room(D), self._packed(D), torch.empty((T,), device="cuda")
        gg.rms_norm(x, D, None, 0, self.master["g1"], EPS, None, 0, n, D, nc, D, ns, ns.stride(0), rstd1, T, D, BF16)
        z, a, (zc, zs) = self._room(H), self._room(H), self._packed(H)
        gg.linear(n, D, self.whole("w1", r), D, "nk", None, "silu", None, 0, a, H, z, H, T, H, D, BF16)
        gg.pack8(z, H, zc, H, zs, zs.stride(0), T, H, BF16)
        m, h, y, rstd2 = self._room(D), self._room(D), self._room(D), torch.empty((T,), device="cuda")
        gg.linear(a, H, self.whole("w2", r), H, "nk", None, "none", None, 0, m, D, None, 0, T, D, H, BF16)
        gg.rms_norm(m, D, x, D, self.master["g2"], EPS, h, D, y, D, None, 0, None, 0, rstd2, T, D, BF16)
        return y, dict(nc=nc, ns=ns, rstd1=rstd1, zc=zc, zs=zs, h=h, rstd2=rstd2)

    def backward(self, x, y, kept, batch, r, accumulate):
        """Statistics and losses of rank r's tokens, and the gradient of x; the weights' gradients (+)=."""
        T, D, H, V, k, g, ws = self.T, self.dim, self.hidden, self.vocab, kept, self.grad, self.scratch
        stats, loss = torch.empty((2,), device="cuda"), torch.empty((T,), device="cuda")
        gg.linear_cross_entropy(y, D, self.whole("wv", r), D, "nk", batch["target"], batch["weight"], stats, loss, None,
                                y, D, g["wv"], D, F32, accumulate, ws, T, V, D, BF16)     # dy over y
        dh, dz, dn = self._room(D), self._room(H), self._room(D)
        gg.rms_norm_backward(y, D, k["h"], D, k["rstd2"], self.master["g2"], None, 0, dh, D, g["g2"], F32, accumulate, ws,
                             T, D, BF16)
        gg.linear_backward8(dh, D, k["zc"], H, k["zs"], k["zs"].stride(0), "silu", self.whole("w2", r), H, "nk", dz, H,
                            g["w2"], H, None, F32, accumulate, ws, T, D, H, BF16)
        gg.linear_backward8(dz, H, k["nc"], D, k["ns"], k["ns"].stride(0), "none", self.whole("w1", r), D, "nk", dn, D,
                            g["w1"], D, None, F32, accumulate, ws, T, H, D, BF16)
        gg.rms_norm_backward(dn, D, x, D, k["rstd1"], self.master["g1"], dh, D, dn, D, g["g1"], F32, accumulate, ws,
                             T, D, BF16)
        return stats, loss, dn

    def step(self, batch, lr=1e-3):
        """One step; the weighted loss, and every rank's losses and gradients of x."""
        self.gather()
        stats, losses, dx = torch.zeros((2,), device="cuda"), [], []
        for r in range(self.W):
            b = {k: v[r] for k, v in batch.items()}
            y, kept = self.forward(b["x"], r)
            s, loss, d = self.backward(b["x"], y, kept, b, r, accumulate=r > 0)
            stats += s
            losses.append(loss)
            dx.append(d)
        self.step_count += 1
        gg.adamw(self.table, self.step_count, lr)
        return stats, torch.stack(losses), torch.stack(dx)


def make_batch(model, seed=1, masked=0.25):
    """Tokens of W shards, some of them masked."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    W, T = model.W, model.T
    keep = torch.rand((W, T), generator=gen, device="cuda") >= masked
    return {"x": torch.randn((W, T, model.dim), generator=gen, device="cuda").to(BF16),
            "target": torch.randint(0, model.vocab, (W, T), generator=gen, device="cuda"),
            "weight": keep.float() / keep.sum()}


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--ranks", type=int, default=4)
    args = ap.parse_args()
    model = ShardedBlock(W=args.ranks)
    batch = make_batch(model)
    for k in range(args.steps):
        stats, _, _ = model.step(batch)
        print(f"step {k + 1:3d}  loss {float(stats[0]):.4f}")


if __name__ == "__main__":
    main()
