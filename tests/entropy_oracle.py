"""How exact the vocabulary's losses have to be: a bound that sees more than the worst case does (device-independent)."""
from __future__ import annotations

import torch

# The tensor cores' accumulator truncates, which costs losses 4.5e-7 of their size (relative errors of all tokens'
# losses together) after a contraction of 1024 and 1.1e-6 after 2011: some 5.5e-10 an element, of the longest
# contraction that is one chunk.  Twice that, and a rounding to float32 of each of lse and the loss.
PER_ELEMENT = 2 * 5.5e-10
ROUNDINGS = 2 * 2.0 ** -24


def relative(got, want):
    """The error of all of a vector, relative to its size."""
    got, want = got.double(), want.double()
    return float((got - want).norm() / want.norm())


def loss_bound(chunk: int) -> float:
    return PER_ELEMENT * chunk + ROUNDINGS


def losses64(x, w, target):
    """Losses and lse of hidden states x and weight rows w (V x K), in float64."""
    z = x.double() @ w.double().t()
    lse = torch.logsumexp(z, 1)
    return lse - z.gather(1, target[:, None])[:, 0], lse
