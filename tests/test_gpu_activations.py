"""The activations and their slopes where little is left of them, and where Z is beyond all bounds.

Y is the once-rounded value: relative to itself, not to Z.  The arithmetic is float32 with paired
operations and the GPU's approximate 2^x and 1/x (2^-22 each): relative 2^-19 in all, and the
exponent y of a power 2^y carries 2^-22 |y| of rounding and of its constants, as much of the power.
Z is exact here: the product with a unit matrix.
"""
import math

import pytest
import torch

from tests.test_gpu_linear import BF16, F16, call_linear, half_ulp, out_mat

pytestmark = pytest.mark.gpu

LOW = {"gelu": -13.0, "gelu_tanh": -9.0, "silu": -80.0}     # above: results and powers are normal floats


def exponent(z, act):
    """The size of the exponent (of 2) in an activation's power."""
    if act == "gelu":
        return z * z * 0.7213475
    if act == "gelu_tanh":
        return (2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)).abs() * 1.442695
    return z.abs() * 1.442695


def terms(z, act):
    """Value, and the two terms of the slope, in float64 without cancellation."""
    if act == "gelu":
        phi, cdf = torch.exp(-z * z / 2) / math.sqrt(2 * math.pi), 0.5 * torch.erfc(-z / math.sqrt(2))
        return z * cdf, cdf, z * phi
    if act == "gelu_tanh":
        u2 = 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
        du = 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z)
    else:
        u2, du = z, torch.ones_like(z)
    s, rest = torch.sigmoid(u2), torch.sigmoid(-u2)
    return z * s, s, z * s * rest * du


def points(act, dtype):
    low = LOW[act]
    z = torch.cat([torch.linspace(low, 0, 4000), -torch.logspace(-6, math.log10(-low), 96)])
    return z.to(dtype).cuda()


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("path", ["split", "pair"])
def test_left_tails(act, dtype, path):
    z = points(act, dtype).view(64, 64)
    unit = torch.eye(64, dtype=dtype, device="cuda")
    y = out_mat(64, 64, dtype)
    call_linear(z, unit, "kn", None, act, None, y, None, path)
    z64 = z.double()
    want, _, _ = terms(z64, act)
    off = (2.0 ** -19 + 2.0 ** -22 * exponent(z64, act)) * want.abs()
    assert ((y.double() - want).abs() <= off + half_ulp(want.abs() + off, dtype)).all()


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_slopes_in_the_left_tails(act, dtype):
    import gemm_gather_gb300 as gg
    z = points(act, dtype).view(64, 64)
    dy, dz = torch.ones_like(z), out_mat(64, 64, dtype)
    gg.act_backward(dy, 64, z, 64, dz, 64, act, 64, 64, dtype)
    z64 = z.double()
    _, a, b = terms(z64, act)
    off = (2.0 ** -18 + 2.0 ** -21 * exponent(z64, act)) * (a.abs() + b.abs())  # two terms, one more product
    assert ((dz.double() - (a + b)).abs() <= off + half_ulp((a + b).abs() + off, dtype)).all()


ALL = ["none", "relu", "gelu", "gelu_tanh", "silu"]


@pytest.mark.parametrize("act", ALL)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_beyond_all_bounds(act, dtype):
    """Large, infinite and NaN Z: slopes are 1 to the right, 0 to the left (none: 1) and NaN at NaN (relu: 0),
    through the elementwise gradient, the input gradient's epilogue, and for Y itself."""
    import gemm_gather_gb300 as gg
    big = torch.finfo(dtype).max
    z = torch.zeros((64, 64), dtype=dtype, device="cuda")
    right = torch.tensor([200.0, 3e4, big / 2, big, math.inf], dtype=dtype)
    if dtype == BF16:
        right = torch.cat([right, torch.tensor([1e15, 1.9e19, 4e30]).to(dtype)])
    n = len(right)
    z[3, :n], z[3, 20:20 + n], z[3, 40] = right, -right, math.nan
    unit = torch.eye(64, dtype=dtype, device="cuda")
    ones, dz = torch.ones_like(z), out_mat(64, 64, dtype)
    gg.act_backward(ones, 64, z, 64, dz, 64, act, 64, 64, dtype)
    for path in ("split", "pair"):
        dx = out_mat(64, 64, dtype)
        gg.linear_backward(ones, 64, None, 64, unit, 64, "kn", z, 64, act, dx, 64, None, 0, None, dtype, False, 64, 64, 64,
                           dtype, path=path)
        assert torch.equal(dx[:, :40], dz[:, :40]) and torch.equal(dx[3, 40].isnan(), dz[3, 40].isnan())
    assert (dz[3, :n] == 1).all() and (dz[3, 20:20 + n] == (1 if act == "none" else 0)).all()
    if act == "relu":
        assert dz[3, 40] == 0
    else:
        assert dz[3, 40].isnan() or act == "none"
    # Y: finite operands only reach the product; the largest finite Z
    y, y2 = out_mat(64, 64, dtype), out_mat(64, 64, dtype)
    x = torch.where(z.isfinite(), z, torch.zeros_like(z))
    for path in ("split", "pair"):
        gg.linear(x, 64, unit, 64, "kn", None, act, None, 0, y, 64, None, 0, 64, 64, 64, dtype, path=path)
        assert torch.equal(y[3, :n], x[3, :n])
        assert torch.equal(y[3, 20:20 + n], x[3, 20:20 + n] if act == "none" else torch.zeros_like(x[3, :n]))
    # an infinite or NaN bias reaches Z as it is
    bias = torch.tensor([math.inf, -math.inf, math.nan] + [0.0] * 61, device="cuda")
    gg.linear(x, 64, unit, 64, "kn", bias, act, None, 0, y, 64, y2, 64, 64, 64, 64, dtype)
    assert (y[5, 0] == math.inf) and y[5, 2].isnan() and y2[5, 1] == -math.inf
    want = {"none": -math.inf, "relu": 0.0, "gelu": 0.0}.get(act, math.nan)
    assert y[5, 1].isnan() if math.isnan(want) else y[5, 1] == want
