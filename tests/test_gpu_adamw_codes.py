"""The 8-bit states of AdamW, code by code: what the definition gives in float32, each operation rounded
to nearest, with its hash for the random bits."""
import numpy as np
import pytest
import torch

import gg_inputs
from tests.test_gpu_adamw import BF16, BLOCK, F16, F32, HYPER, make, run

pytestmark = pytest.mark.gpu


def mix32(x):
    x = x.astype(np.uint32)
    x ^= x >> np.uint32(16)
    x = x * np.uint32(0x7FEB352D)
    x ^= x >> np.uint32(15)
    x = x * np.uint32(0x846CA68B)
    return x ^ (x >> np.uint32(16))


def random_bits(n, seed, step, position):
    key = np.array([position], dtype=np.uint32)
    for word in (step, seed, seed >> 32):
        key = mix32(key) ^ np.uint32(word & 0xFFFFFFFF)
    return mix32(np.arange(n, dtype=np.uint32) ^ mix32(mix32(key)))


def blocks(x):
    return np.pad(x, (0, -len(x) % BLOCK)).reshape(-1, BLOCK)


def to_codes(x, r16):
    """The values that the codes of x stand for before scaling, and the scales."""
    b = blocks(np.abs(x))
    frac, power = np.frexp(b.max(1))
    k = np.maximum(np.where(b.max(1) > 0, power - 9 + (frac > 0.875), -118), -118)
    y = (np.abs(x).astype(np.float64) / np.repeat(np.exp2(k.astype(np.float64)), BLOCK)[:len(x)]).astype(np.float32)
    low = y < 0.015625                       # below 2^-6 the step stays 2^-9: the same, on y + 2^-6
    z = np.where(low, y + np.float32(0.015625), y).astype(np.float32)
    cut = ((z.view(np.uint32) + (r16.astype(np.uint32) << np.uint32(4))) & np.uint32(0xFFF00000)).view(np.float32)
    return np.copysign(np.where(low, cut - np.float32(0.015625), cut), x), np.exp2(k).astype(np.float32)


@pytest.mark.parametrize("param,grad,copy", [(F32, BF16, BF16), (BF16, BF16, None), (F32, F32, None), (F16, F16, None)])
@pytest.mark.parametrize("shift", [0, 1])
def test_codes_and_scales(param, grad, copy, shift):
    step, seed = 7, (5 << 32) + 11
    sizes = [70000, 257, 3000000]
    ts = [make(n, param, grad, 8, copy, shift, gen=gg_inputs.generator(n + shift)) for n in sizes]
    f = np.float32
    b1, b2 = f(HYPER["beta1"]), f(HYPER["beta2"])
    o1, o2 = f(1.0 - HYPER["beta1"]), f(1.0 - HYPER["beta2"])
    want = []
    for position, t in enumerate(ts):
        n = t["param"].numel()
        g = t["grad"].float().cpu().numpy() * f(0.37)
        m, u = ((t[k].view(torch.float8_e4m3fn).float() * t[k + "_scale"].repeat_interleave(BLOCK)[:n]).cpu().numpy()
                for k in ("m", "v"))
        m = m * b1 + g * o1
        v = (u * u) * b2 + (g * g) * o2
        r = random_bits(n, seed, step, position)
        want.append([to_codes(m, r & np.uint32(0xFFFF)), to_codes(np.sqrt(v), r >> np.uint32(16))])
    run(ts, step, 8, gs=0.37, seed=seed)
    for t, states in zip(ts, want):
        for k, (codes, scales) in zip(("m", "v"), states):
            assert np.array_equal(t[k + "_scale"].cpu().numpy(), scales)
            got = t[k].view(torch.float8_e4m3fn).float().cpu().numpy()
            assert np.array_equal(got, codes), (k, int((got != codes).sum()))
