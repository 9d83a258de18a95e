"""The linear layer at its edges: tiles that a matrix fills in part, weight gradients on their own.

Integer-valued operands make every product and partial sum an exact float32 integer, so results have
to be equal bit for bit.
"""
import pytest
import torch

import gg_inputs
from tests.test_gpu_linear import (BF16, F16, F32, FILL, call_backward, call_linear, mat, out_mat, padding, status_ok,
                                   weight64)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K", [(1, 1, 2048), (1, 64, 4096), (3, 33, 4000), (16, 129, 1000), (40, 160, 1500),
                                   (60, 257, 1024)])
def test_split_tiles_with_warps_past_the_last_feature(M, N, K):
    """Tiles split between the CTAs of a cluster, of which whole warps have no feature: 20 launches
    back to back, each with its CTAs leaving while the next starts."""
    gen = gg_inputs.generator(M + N)
    x, w = mat(M, K, BF16, gen, ints=True), mat(N, K, BF16, gen, ints=True)
    ys = [out_mat(M, N, BF16, 3) for _ in range(20)]
    for y in ys:
        call_linear(x, w, "nk", None, "none", None, y, None, "split")
    want = (x.double() @ w.double().t()).to(BF16)
    for y in ys:
        assert torch.equal(y, want) and (padding(y) == FILL).all()
    status_ok()


@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("M,N,K", [(1100, 96, 515), (640, 257, 300), (900, 129, 70), (2048, 256, 512)])
def test_split_float32_gradients_past_the_last_feature_and_token(M, N, K, layout):
    """Weight gradients whose tokens are split between CTA pairs, added to what the gradient holds."""
    gen = gg_inputs.generator(M + N + K)
    dz, x = mat(M, N, F16, gen, ints=True), mat(M, K, F16, gen, ints=True)
    dw = out_mat(*((K, N) if layout == "kn" else (N, K)), F32, 1)
    dw.zero_()
    for _ in range(20):
        call_backward(dz, x, x, layout, None, "none", None, dw, None, True, "pair")
    g = x.double().t() @ dz.double()
    assert torch.equal(dw.double(), 20 * (g if layout == "kn" else g.t()))
    assert (padding(dw) == FILL).all()
    status_ok()


@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (27, 3584, 512), (300, 1024, 1024), (700, 640, 2048)])
def test_same_bits_wherever_the_operands_lie(M, N, K):
    """The same matrices 16 and 112 bytes behind a 128-byte line: equal sums, bit for bit, of values whose
    sum depends on its order."""
    gen = gg_inputs.generator(M)

    def copies(t):
        out = []
        for shift in (0, 8, 56):
            buf = torch.empty(t.numel() + 64, dtype=t.dtype, device="cuda")
            assert buf.data_ptr() % 128 == 0
            out.append(buf[shift:shift + t.numel()].view(t.shape).copy_(t))
        return out

    xs, ws, dzs = copies(mat(M, K, F16, gen)), copies(mat(N, K, F16, gen)), copies(mat(M, N, F16, gen))
    got = []
    for x, w, dz in zip(xs, ws, dzs):
        y, dx, dw, db = out_mat(M, N, F16), out_mat(M, K, F16), out_mat(N, K, F32), torch.zeros(N, device="cuda")
        call_linear(x, w, "nk", None, "none", None, y, None)
        call_backward(dz, x, w, "nk", None, "none", dx, dw, db, False)
        got.append((y, dx, dw, db))
    for other in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got[0], other))
    status_ok()


# One gradient at a time, where nothing else shares the launch: tiles of 128 and 256 tokens, whole, or their
# contraction split between 2 and 4 CTA pairs (weight gradients on "pair": 128 whole, 128 by 2, 128 by 4, 256 by 2, 256 by
# 4, 256 whole), with ragged edges on both sides.
GRADIENTS = [(70, 96, 130), (2048, 515, 1030), (640, 257, 300), (5000, 1030, 1030), (900, 300, 1030), (300, 3500, 2050)]


@pytest.mark.parametrize("path", ["split", "pair", "auto"])
@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("grad", [F16, BF16, F32])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("M,N,K", GRADIENTS)
def test_weight_gradients_alone(M, N, K, accumulate, grad, layout, path):
    gen = gg_inputs.generator(M + N + K)
    dtype = F16 if grad == F32 else grad
    dz, x = mat(M, N, dtype, gen, ints=True), mat(M, K, dtype, gen, ints=True, pad=8)
    dw = out_mat(*((K, N) if layout == "kn" else (N, K)), grad, 3)
    dw.copy_(gg_inputs.integers(tuple(dw.shape), -2, 2, F32, gen))
    before = dw.double()
    call_backward(dz, x, x, layout, None, "none", None, dw, None, accumulate, path)
    g = x.double().t() @ dz.double()
    assert torch.equal(dw, ((g if layout == "kn" else g.t()) + before * accumulate).to(grad))
    assert (padding(dw) == FILL).all()
    status_ok()


@pytest.mark.parametrize("path", ["split", "pair", "auto"])
@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("M,N,K", GRADIENTS + [(256, 4100, 1000), (600, 8000, 700)])
def test_input_gradients_alone(M, N, K, layout, path):
    gen = gg_inputs.generator(M + N + K)
    dz, z = mat(M, N, BF16, gen, ints=True), mat(M, K, BF16, gen, ints=True, pad=8)
    w = mat(*((K, N) if layout == "kn" else (N, K)), BF16, gen, ints=True)
    dx = out_mat(M, K, BF16, 5)
    call_backward(dz, z, w, layout, z, "relu", dx, None, None, False, path)
    assert torch.equal(dx, ((dz.double() @ weight64(w, layout).t()) * (z > 0)).to(BF16))
    assert (padding(dx) == FILL).all()
    status_ok()
