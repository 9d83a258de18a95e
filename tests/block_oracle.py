"""The norm, the 8-bit activations and the vocabulary's cross entropy in float64, from their formulas,
and the matrices their tests are made of (device-independent; no code of the library)."""
from __future__ import annotations

import math

import torch

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
F64 = torch.float64
BLOCK = 128
MANT = {F16: 10, BF16: 7, F32: 23}
TOP = {F16: 65504.0, BF16: 3.3895313892515355e38}
FILL = 77.0           # what columns beyond a row hold before and after


def power_of_two(e):
    return ((e.to(torch.int64) + 1023) << 52).view(F64)


def half_ulp(x, dtype):
    ax = torch.clamp_min(x.abs(), 2.0 ** (-14 if dtype == F16 else -126))
    return torch.exp2(torch.floor(torch.log2(ax)) - MANT[dtype] - 1)


def pack(x):
    """(values of the codes, scales) of a matrix in 16 bits, by e4m3's steps: 2^-9 below 2^-6, an eighth
    of the power of two above; ties to even.  What is not finite: NaN, outside the scale."""
    M, N = x.shape
    x = x.double()
    fine = torch.isfinite(x)
    whole = torch.zeros((M, -(-N // BLOCK) * BLOCK), dtype=F64, device=x.device)
    whole[:, :N] = torch.where(fine, x, 0.0)
    top = whole.abs().view(M, -1, BLOCK).amax(2)
    frac, power = torch.frexp(top)
    power = torch.where(frac == 0, -200, power)     # nothing but zeros: the least scale
    scale = power_of_two(torch.clamp(power - 9 + (frac > 0.875).to(power.dtype), min=-118))
    y = whole[:, :N] / scale.repeat_interleave(BLOCK, 1)[:, :N]
    quantum = power_of_two(torch.clamp(torch.frexp(y).exponent - 4, min=-9))
    return torch.where(fine, torch.round(y / quantum) * quantum, math.nan), scale


def values(codes, scales):
    """What codes (float8_e4m3fn, or their values) and scales stand for."""
    s = scales.double().repeat_interleave(BLOCK, 1)[:, :codes.shape[1]]
    return codes.double() * s


def act64(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return z * 0.5 * (1 + torch.erf(z / math.sqrt(2)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if act == "silu":
        return z * torch.sigmoid(z)
    return z


def slope64(z, act):
    if act == "none":
        return torch.ones_like(z)
    if act == "relu":
        return (z > 0).double()
    h = 1e-5
    return (act64(z + h, act) - act64(z - h, act)) / (2 * h)


def room(rows, cols, dtype, pad=0, shift=0, device="cuda", unit=8):
    """rows x cols at `shift` elements from a 16-byte boundary, with a pitch of whole 16 bytes + pad."""
    ld = (cols + unit - 1) // unit * unit + pad
    buf = torch.full((rows * ld + shift,), FILL, dtype=F32, device=device).to(dtype)
    return buf[shift:].as_strided((rows, cols), (ld, 1), shift)


def put(x, dtype, pad=0, shift=0, device="cuda"):
    out = room(*x.shape, dtype, pad, shift, device)
    out.copy_(x.to(dtype))
    return out


def rest(view):
    """What of a view's storage is not its own."""
    whole = view.as_strided((view.untyped_storage().nbytes() // view.element_size(),), (1,), 0)
    own = torch.zeros(whole.shape, dtype=torch.bool, device=view.device)
    own.as_strided(view.shape, view.stride(), view.storage_offset()).fill_(True)
    return whole[~own]


def untouched(view):
    r = rest(view).float()
    return bool((r == torch.full_like(r, FILL).to(view.dtype).float()).all())
