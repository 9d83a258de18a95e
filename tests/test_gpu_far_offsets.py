"""Matrices of more than 2^31 elements: the last rows of what the norm, the 8-bit activations, a layer's gradients
from them and the cross entropy read and write."""
import pytest
import torch

import gemm_gather_gb300 as gg
from tests import block_oracle as o
from tests.block_oracle import BF16, F32
from tests.test_gpu_norm import backward, check_norm, gradients64, norm

pytestmark = pytest.mark.gpu

M, N = 270000, 8192                     # 2.2e9 elements
LAST = slice(M - 40, M)
U8, E4M3 = torch.uint8, torch.float8_e4m3fn


def big(seed, dtype=BF16, ld=N):
    g = torch.Generator(device="cuda").manual_seed(seed)
    buf = torch.empty((M, ld), dtype=dtype, device="cuda")
    for r in range(0, M, 30000):
        part = buf[r:r + 30000]
        part.copy_(torch.randn(part.shape, generator=g, device="cuda"))
    return buf[:, :N]


@pytest.mark.parametrize("ld", [N, N + 1])
def test_norm(ld):
    x, r = big(1, ld=ld), big(2, ld=ld)
    w = torch.randn((N,), device="cuda").to(BF16)
    h, y = (torch.empty((M, ld), dtype=BF16, device="cuda")[:, :N] for _ in range(2))
    codes, scales = torch.empty((M, N), dtype=U8, device="cuda"), torch.empty((M, N // 128), device="cuda")
    rstd = torch.empty((M,), device="cuda")
    norm(x, r, w, h=h, y=y, codes=codes.view(E4M3), scales=scales, rstd=rstd)
    for rows in (slice(0, 40), LAST):
        check_norm(x[rows], r[rows], w, 1e-6, h[rows], y[rows], codes[rows].view(E4M3), scales[rows], rstd[rows])
    dh, dw = x, torch.empty((N,), device="cuda")       # (x is not needed any more)
    backward(y, h, rstd, w, r, dh, dw, workspace=torch.empty((608 * N * 4,), dtype=U8, device="cuda"))
    for rows in (slice(0, 40), LAST):
        want, size, _, _ = gradients64(y[rows], h[rows], rstd[rows], w, r[rows])
        assert ((dh[rows].double() - want).abs() <= size * (N / 512 + 52) * 2.0 ** -24 + o.half_ulp(want, BF16) * 1.01).all()
    ww, size = torch.zeros((N,), dtype=torch.float64, device="cuda"), torch.zeros((N,), dtype=torch.float64, device="cuda")
    for k in range(0, M, 30000):
        t = y[k:k + 30000].double() * h[k:k + 30000].double() * rstd[k:k + 30000].double()[:, None]
        ww += t.sum(0)
        size += t.abs().sum(0)
    # at most M / 304 rows of a block one after the other, and the blocks' sums
    assert ((dw.double() - ww).abs() <= size * (M / 304 + 32) * 2.0 ** -24).all()


def test_packing_and_a_layers_gradients():
    P = 64                                              # the layer's outputs
    x = big(3)
    codes, scales = torch.empty((M, N), dtype=U8, device="cuda"), torch.empty((M, N // 128), device="cuda")
    gg.pack8(x, N, codes, N, scales, N // 128, M, N, BF16)
    for rows in (slice(0, 40), LAST):
        c, s = o.pack(x[rows])
        assert torch.equal(codes[rows].view(E4M3).double(), c) and torch.equal(scales[rows].double(), s)
    out = x
    gg.unpack8(codes, N, scales, N // 128, "relu", out, N, M, N, BF16)
    for rows in (slice(0, 40), LAST):
        want = torch.clamp_min(o.values(codes[rows].view(E4M3), scales[rows]), 0).to(BF16)
        assert torch.equal(out[rows], want)
    g = torch.Generator(device="cuda").manual_seed(4)
    dz = torch.randn((M, P), generator=g, device="cuda").to(BF16)
    w = (torch.randn((P, N), generator=g, device="cuda") * P ** -0.5).to(BF16)
    dx, dw, db = x, torch.empty((P, N), device="cuda"), torch.empty((P,), device="cuda")
    room = torch.empty((gg.linear_backward8_workspace(M, N) // 2,), dtype=U8, device="cuda")
    gg.linear_backward8(dz, P, codes, N, scales, N // 128, "relu", w, N, "nk", dx, N, dw, N, db, F32, False, room, M, P, N, BF16)
    for rows in (slice(0, 40), LAST):
        p = o.values(codes[rows].view(E4M3), scales[rows])
        want = (dz[rows].double() @ w.double()) * (p > 0)
        bound = (dz[rows].double().abs() @ w.double().abs()) * P * 2.0 ** -23
        assert ((dx[rows].double() - want).abs() <= bound + o.half_ulp(want, BF16) * 1.01).all()
    cols = torch.tensor([0, 127, 4000, N - 1], device="cuda")
    v = torch.clamp_min(codes.view(E4M3)[:, cols].double() * scales[:, cols // 128].double(), 0)
    want, size = dz.double().t() @ v, dz.double().abs().t() @ v
    # truncating sums of 896 tokens, rounded ones of those
    assert ((dw[:, cols].double() - want).abs() <= size * (896 + M / 896) * 2.0 ** -23).all()
    assert ((db.double() - dz.double().sum(0)).abs() <= dz.double().abs().sum(0) * (M / 64 + 16) * 2.0 ** -24).all()


def test_cross_entropy():
    T, V, K = 70000, 33000, 64                          # the piece's gradient: 2.3e9 elements
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn((T, K), generator=g, device="cuda").to(BF16)
    w = (torch.randn((V, K), generator=g, device="cuda") * 2 * K ** -0.5).to(BF16)
    target = torch.randint(0, V, (T,), generator=g, device="cuda")
    weight = torch.rand((T,), generator=g, device="cuda") + 0.1
    stats, loss, lse = torch.empty(2, device="cuda"), torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    dx, dw = torch.empty_like(x), torch.empty((V, K), device="cuda")
    piece = 33024
    room = torch.empty((gg.linear_cross_entropy_workspace(T, V, K, piece),), dtype=U8, device="cuda")
    gg.linear_cross_entropy(x, K, w, K, "nk", target, weight, stats, loss, lse, dx, K, dw, K, F32, False, room, T, V, K, BF16,
                            piece=piece)
    del room
    x64, w64 = x.double(), w.double()
    for rows in (slice(0, 200), slice(T - 200, T)):
        z = x64[rows] @ w64.t()
        want = torch.logsumexp(z, 1)
        bz = (x64[rows].abs() @ w64.abs().t()).amax(1) * K * 2.0 ** -23 + 2.0 ** -20 + want.abs() * 2.0 ** -23
        assert ((lse[rows].double() - want).abs() <= bz).all()
        assert ((loss[rows].double() - want + z.gather(1, target[rows, None])[:, 0]).abs() <= 2 * bz).all()
        tw = weight[rows].double()[:, None]
        dz = tw * (torch.exp(z - want[:, None]) - torch.zeros_like(z).scatter_(1, target[rows, None], 1.0))
        want = dz @ w64
        bound = (dz.abs() * (2.0 ** -8 + 2.0 ** -11)) @ w64.abs() + (dz.abs() @ w64.abs()) * (V * 2.0 ** -23)
        assert ((dx[rows].double() - want).abs() <= bound + o.half_ulp(want, BF16) * 1.01).all()
    entries = torch.tensor([0, 1, 16000, V - 200, V - 1], device="cuda")
    p = torch.exp(x64 @ w64[entries].t() - lse.double()[:, None])
    dz = weight.double()[:, None] * (p - (target[:, None] == entries).double())
    want = dz.t() @ x64
    # dZ's rounding, and a float32 sum's of 70000 tokens
    bound = (dz.abs() * (2.0 ** -8 + 2.0 ** -11)).t() @ x64.abs() + (dz.abs().t() @ x64.abs()) * ((896 + T / 896) * 2.0 ** -23)
    assert ((dw[entries].double() - want).abs() <= bound).all()
