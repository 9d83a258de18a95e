"""Activations in 8 bits: codes and scales bit by bit, what they stand for, and a linear layer's gradients
from them.

linear_backward8 is linear_backward on the 16-bit matrices that the codes stand for: the same kernels, tiles
and sums, so with both given the same bits come out, and both are within linear_backward's own tolerance of
float64 (the float32 sum's bound, the slope's own arithmetic of 2^-20, X's one rounding of half an ulp, and
half an ulp of the output).  A float32 dW of a smooth activation is that of X in two parts: X is off by half an
ulp of the second one, 2^-9 (2^-12 in float16, or its least step) of half an ulp of the first.
"""
import math

import pytest
import torch

import gemm_gather_gb300 as gg
from gemm_gather_gb300 import _lib
from tests import block_oracle as o
from tests.block_oracle import BF16, F16, F32

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


def codes_room(M, N, pad=0, shift=0):
    ld = (N + 15) // 16 * 16 + pad
    buf = torch.full((M * ld + shift,), 3, dtype=torch.uint8, device="cuda")
    return buf[shift:].as_strided((M, N), (ld, 1), shift).view(E4M3)


def packed(x, pad=0, shift=0):
    M, N = x.shape
    codes, scales = codes_room(M, N, pad, shift), o.room(M, -(-N // 128), F32, pad, 0)
    gg.pack8(x, x.stride(0), codes, codes.stride(0), scales, scales.stride(0), M, N, x.dtype)
    return codes, scales


def check_packed(x, codes, scales):
    c, s = o.pack(x)
    assert torch.equal(scales.double(), s)
    got = codes.double()
    assert torch.equal(got.isnan(), c.isnan()) and torch.equal(got.nan_to_num(), c.nan_to_num())
    assert o.untouched(scales) and bool((o.rest(codes.view(torch.uint8)) == 3).all())


def spread(M, N, dtype, seed=0):
    """Normal values of many sizes: blocks of very different tops, some elements far below their block's."""
    g = torch.Generator().manual_seed(seed + M + 3 * N)
    x = torch.randn((M, N), generator=g) * torch.exp2(torch.randint(-12, 9, (M, N), generator=g).float())
    return x * torch.exp2(torch.randint(-4, 5, (M, 1), generator=g).float())


@pytest.mark.parametrize("M,N", [(1, 1), (1, 8192), (3, 127), (5, 128), (7, 129), (100, 1523), (777, 1000), (2000, 260)])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("pad,shift", [(0, 0), (1, 0), (0, 3)])
def test_pack(M, N, dtype, pad, shift):
    x = o.put(spread(M, N, dtype), dtype, pad, shift)
    codes, scales = packed(x, pad, shift)
    check_packed(x, codes, scales)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("pad", [0, 1])
def test_pack_every_value(dtype, pad):
    """All 65536 patterns of the type, in blocks of one exponent, and next to the scale's borders."""
    x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(dtype).view(512, 128)
    mixed = x.reshape(-1)[torch.randperm(65536, generator=torch.Generator().manual_seed(1))].view(512, 128)
    tops = torch.tensor([448.0, 449.0, 450.0, 447.0, 224.0, 225.0, 223.0, 1.75, 1.7578125, 1.7421875, 2.0 ** -14, 0.0])
    border = (torch.rand((12, 128), generator=torch.Generator().manual_seed(2)) * 2 - 1) * tops[:, None]
    border[:, 77] = tops
    for m in (x, mixed, border):
        y = o.put(m.float(), dtype, pad)
        y.copy_(m.to(dtype))
        codes, scales = packed(y)
        check_packed(y, codes, scales)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,N,pad,shift", [(1, 1, 0, 0), (37, 1000, 0, 0), (64, 129, 1, 0), (50, 1523, 0, 3)])
def test_unpack(M, N, pad, shift, dtype, act):
    x = o.put(torch.randn((M, N), generator=torch.Generator().manual_seed(N)) * 2, dtype)
    codes, scales = packed(x, pad, shift)
    out = o.room(M, N, dtype, pad, shift)
    gg.unpack8(codes, codes.stride(0), scales, scales.stride(0), act, out, out.stride(0), M, N, dtype)
    v = o.values(codes, scales)
    want = o.act64(v, act)
    if act in ("none", "relu"):
        assert torch.equal(out.double(), want.to(dtype).double())
    assert ((out.double() - want).abs() <= 2.0 ** -20 * v.abs() + o.half_ulp(want, dtype) * 1.01).all()
    assert o.untouched(out)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_unpack_every_code_and_the_largest_values(dtype):
    c = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(2, 128).repeat(4, 1).cuda().view(E4M3)
    scales = torch.tensor([[1.0], [1.0], [0.25], [0.25], [2.0 ** -16], [2.0 ** -16], [128.0], [128.0]], device="cuda")
    out = torch.empty((8, 128), dtype=dtype, device="cuda")
    gg.unpack8(c, 128, scales, 1, "none", out, 128, 8, 128, dtype)
    want = o.values(c, scales).to(dtype)
    assert torch.equal(out.isnan(), want.isnan()) and torch.equal(out.nan_to_num(), want.nan_to_num())
    # a rounding up into 8 bits passes the type's range: its largest number comes back
    top = o.TOP[dtype]
    x = torch.full((1, 128), top, dtype=dtype, device="cuda")
    x[0, 1], x[0, 2], x[0, 3] = -top, 0.0, float("inf")
    codes, scales = packed(x)
    out = torch.empty_like(x)
    gg.unpack8(codes, codes.stride(0), scales, scales.stride(0), "none", out, 128, 1, 128, dtype)
    assert out[0, 0] == top and out[0, 1] == -top and out[0, 2] == 0 and out[0, 3].isnan()


# ---- a linear layer's gradients ---------------------------------------------------------------------
def backward8(dz, codes, scales, act, w, layout, dx, dw, db, acc, K, path="auto", workspace=None):
    ld = lambda t: t.stride(0) if t is not None else 0   # noqa: E731
    M, N = dz.shape
    need = gg.linear_backward8_workspace(M, K)
    room = torch.full((need + 32,), 0xEE, dtype=torch.uint8, device="cuda") if workspace is None else workspace
    gdt = dw.dtype if dw is not None else F32
    gg.linear_backward8(dz, ld(dz), codes, ld(codes), scales, ld(scales), act, w, ld(w), layout, dx, ld(dx), dw, ld(dw),
                        db, gdt, acc, room, M, N, K, dz.dtype, path=path, workspace_bytes=need)
    if workspace is None:
        assert (room[need:] == 0xEE).all()


def layer(M, N, K, dtype, layout, seed=0, pad=0):
    g = torch.Generator().manual_seed(seed + M + N + K)
    p = o.put(torch.randn((M, K), generator=g), dtype)
    w = torch.randn((K, N) if layout == "kn" else (N, K), generator=g) * K ** -0.5
    dz = torch.randn((M, N), generator=g) * 0.25
    codes, scales = packed(p, pad)
    return codes, scales, o.put(w, dtype), o.put(dz, dtype)


SHAPES = [(1, 64, 64), (16, 200, 72), (27, 130, 1000), (100, 1000, 129), (300, 96, 520), (777, 1000, 1523), (1024, 512, 2048)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_backward8(M, N, K, layout, dtype):
    i = SHAPES.index((M, N, K))
    act, acc = ACTS[(i + (layout == "kn")) % 5], i % 2 == 0
    gdt = F32 if (i + (dtype is F16)) % 2 else dtype
    codes, scales, w, dz = layer(M, N, K, dtype, layout, pad=i % 2)
    p = o.values(codes, scales).to(dtype)          # held in 16 bits without loss at these sizes
    for path in ("auto", "split", "pair"):
        dx, dw = o.room(M, K, dtype), torch.randn(w.shape, device="cuda").to(gdt)
        db = torch.randn((N,), device="cuda").to(gdt)
        dw0, db0 = dw.clone(), db.clone()
        backward8(dz, codes, scales, act, w, layout, dx, dw, db, acc, K, path)
        x = o.room(M, K, dtype)
        gg.unpack8(codes, codes.stride(0), scales, scales.stride(0), act, x, x.stride(0), M, K, dtype)
        # the same through 16-bit matrices: equal bits
        z = o.put(p, dtype)
        dx2, dw2, db2 = o.room(M, K, dtype), dw0.clone(), db0.clone()
        gg.linear_backward(dz, dz.stride(0), x, x.stride(0), w, w.stride(0), layout, z if act != "none" else None, z.stride(0),
                           act, dx2, dx2.stride(0), dw2, dw2.stride(0), db2, gdt, acc, M, N, K, dtype, path=path)
        two = gdt is F32 and act not in ("none", "relu")
        assert torch.equal(dx.view(torch.int16), dx2.view(torch.int16)) and torch.equal(db, db2)
        assert two or torch.equal(dw, dw2)
        # and float64
        p64, w64, dz64 = p.double(), w.double() if layout == "kn" else w.double().t(), dz.double()
        slope = o.slope64(p64, act)
        want = (dz64 @ w64.t()) * slope
        bound = (dz64.abs() @ w64.abs().t()) * 1.13 * (N * 2.0 ** -23 + 2.0 ** -19) + o.half_ulp(want, dtype) * 1.01
        assert ((dx.double() - want).abs() <= bound).all()
        x64 = o.act64(p64, act)
        part = 2.0 ** (-12 if dtype is F16 else -9) if two else 1.0
        xe = x64.abs() * ((M + 1) * 2.0 ** -23) + o.half_ulp(x64, dtype) * 1.01 * part + 2.0 ** -20 * p64.abs()
        if two and dtype is F16:
            xe = xe + 2.0 ** -25
        want, bound = x64.t() @ dz64, xe.t() @ dz64.abs()
        if layout == "nk":
            want, bound = want.t(), bound.t()
        if acc:
            want, bound = want + dw0.double(), bound + dw0.double().abs() * 2.0 ** -23
        assert ((dw.double() - want).abs() <= bound + o.half_ulp(want, gdt) * 1.01).all()
        assert o.untouched(dx)


def test_backward8_parts_alone():
    M, N, K = 130, 264, 520
    codes, scales, w, dz = layer(M, N, K, BF16, "nk")
    dx, dw, db = o.room(M, K, BF16), torch.empty(w.shape, device="cuda"), torch.empty((N,), device="cuda")
    for path in ("split", "pair"):
        backward8(dz, codes, scales, "gelu", w, "nk", dx, dw, db, False, K, path)
        dx1, dw1, db1 = o.room(M, K, BF16), torch.empty_like(dw), torch.empty_like(db)
        none = torch.empty((0,), dtype=torch.uint8, device="cuda")
        gg.linear_backward8(dz, dz.stride(0), codes, codes.stride(0), scales, scales.stride(0), "gelu", w, w.stride(0), "nk",
                            dx1, dx1.stride(0), None, 0, None, F32, False, None, M, N, K, BF16, path=path)
        backward8(dz, codes, scales, "gelu", None, "nk", None, dw1, None, False, K, path)
        gg.linear_backward8(dz, dz.stride(0), None, 0, None, 0, "gelu", None, 0, "nk", None, 0, None, 0, db1, F32, False,
                            none, M, N, K, BF16, path=path)
        if path == "split":   # (pairs walk both products together, with other tiles than each alone)
            assert torch.equal(dx.view(torch.int16), dx1.view(torch.int16)) and torch.equal(dw, dw1)
        assert torch.equal(db, db1)
        # dX alone without an activation reads no codes
        dx2 = o.room(M, K, BF16)
        gg.linear_backward8(dz, dz.stride(0), None, 0, None, 0, "none", w, w.stride(0), "nk", dx2, dx2.stride(0), None, 0,
                            None, F32, False, None, M, N, K, BF16, path=path)
        want = dz.double() @ w.double()
        assert ((dx2.double() - want).abs() <= (dz.double().abs() @ w.double().abs()) * N * 2.0 ** -23
                + o.half_ulp(want, BF16) * 1.01).all()


def test_backward8_empty_sizes():
    w = torch.ones((8, 16), dtype=BF16, device="cuda")
    dw, db = torch.full((8, 16), 3.0, device="cuda"), torch.full((8,), 4.0, device="cuda")
    gg.linear_backward8(None, 8, None, 16, None, 1, "silu", w, 16, "nk", None, 16, dw, 16, db, F32, True, None, 0, 8, 16, BF16)
    assert (dw == 3).all() and (db == 4).all()
    gg.linear_backward8(None, 8, None, 16, None, 1, "silu", w, 16, "nk", None, 16, dw, 16, db, F32, False, None, 0, 8, 16, BF16)
    assert (dw == 0).all() and (db == 0).all()
    codes, scales = packed(torch.randn((5, 16), device="cuda").to(BF16))
    dx = torch.full((5, 16), 9.0, dtype=BF16, device="cuda")
    gg.linear_backward8(None, 8, codes, codes.stride(0), scales, 1, "silu", None, 16, "nk", dx, 16, None, 16, None, F32, False,
                        None, 5, 0, 16, BF16)
    assert (dx == 0).all()


def test_backward8_infinite_and_nan_codes():
    """A NaN code is NaN in its token's dX element and in its column of dW, and nowhere else."""
    M, N, K = 40, 64, 256
    codes, scales, w, dz = layer(M, N, K, BF16, "nk")
    codes.view(torch.uint8)[7, 130] = 0x7F
    for path in ("split", "pair"):
        dx, dw = o.room(M, K, BF16), torch.empty(w.shape, device="cuda")
        backward8(dz, codes, scales, "silu", w, "nk", dx, dw, None, False, K, path)
        bad = torch.zeros((M, K), dtype=torch.bool, device="cuda")
        bad[7, 130] = True
        assert torch.equal(dx.isnan(), bad)
        assert dw[:, 130].isnan().all() and dw.isnan().sum() == N


def test_backward8_reports_a_wait_that_gave_up():
    codes, scales, w, dz = layer(300, 256, 512, BF16, "nk")
    dx, dw = o.room(300, 512, BF16), torch.empty(w.shape, device="cuda")
    room = torch.empty((gg.linear_backward8_workspace(300, 512),), dtype=torch.uint8, device="cuda")
    status = torch.zeros((1,), dtype=torch.int32, device="cuda")

    def call(word):
        gg.linear_backward8(dz, dz.stride(0), codes, codes.stride(0), scales, scales.stride(0), "silu", w, w.stride(0), "nk",
                            dx, dx.stride(0), dw, dw.stride(0), None, F32, False, room, 300, 256, 512, BF16, status=word)
    gg.set_wait_limit_ns(20_000_000)
    gg.debug_inject_stall(True)
    try:
        call(status)
        torch.cuda.synchronize()
    finally:
        gg.debug_inject_stall(False)
        gg.set_wait_limit_ns(0)
    assert int(status) == _lib.GG_ERR_TIMEOUT
    status.zero_()
    call(status)
    first = dx.clone(), dw.clone()
    call(status)
    assert int(status) == 0 and torch.equal(first[0], dx) and torch.equal(first[1], dw) and math.isfinite(float(dw.sum()))
