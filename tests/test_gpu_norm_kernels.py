"""Every kernel that the norm and its gradients choose between by a row's length and the number of rows, each
named from what a call launches: vectors a thread, rows in flight, rows of whole vectors or not.  The bounds are
test_gpu_norm.py's: a thread adds up to 32 squares or products here too."""
import numpy as np
import pytest
import torch

from tests import block_oracle as o
from tests.block_oracle import BF16, F16, F32
from tests.launched import variants
from tests.test_gpu_norm import (backward, bits, check_gradients, check_norm, codes_room, gradients64, make, make_backward, norm)

pytestmark = pytest.mark.gpu


# M, N, vectors a thread, rows of whole vectors
@pytest.mark.parametrize("M,N,vpt,whole", [(2000, 700, 2, 0), (2000, 704, 2, 1), (4000, 515, 2, 0), (2500, 2043, 4, 0),
                                           (2500, 2048, 4, 1), (700, 8192, 4, 1), (700, 8189, 4, 0), (100, 1523, 1, 0)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_forward(M, N, vpt, whole, dtype):
    for residual in (True, False):
        x, r, w = make(M, N, dtype, wdtype=F32 if residual else dtype, residual=residual)
        h, y = o.room(M, N, dtype), o.room(M, N, dtype, pad=8)
        codes, scales = codes_room(M, N), o.room(M, -(-N // 128), F32, pad=1)
        rstd = torch.empty((M,), device="cuda")

        def call():
            norm(x, r, w, h=h, y=y, codes=codes, scales=scales, rstd=rstd)
        call()
        check_norm(x, r, w, 1e-6, h, y, codes, scales, rstd)
        assert o.untouched(h) and o.untouched(y) and o.untouched(scales)
        assert bool((o.rest(codes.view(torch.uint8)) == 3).all())
        assert [k for _, k, _ in variants(call, "norm_kernel")] == [(int(dtype is BF16), vpt, int(residual), whole)]


# M, N, vectors a thread, rows in flight with and without what arrives along the residual, rows of whole vectors
# (rows that are not copied ahead are read by one kernel, whole vectors or not)
@pytest.mark.parametrize("M,N,vpt,depth,whole", [
    (2500, 2048, 4, (2, 3), 1), (700, 8192, 4, (2, 3), 1), (2500, 2043, 4, (2, 3), 0), (1300, 2600, 4, (2, 3), 1),
    (700, 8189, 4, (2, 3), 0), (311, 8192, 4, (1, 1), 0), (2000, 700, 2, (1, 1), 0), (4000, 515, 2, (1, 1), 0),
    (100, 1523, 1, (1, 1), 0)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_backward(M, N, vpt, depth, whole, dtype):
    for through in (True, False):
        dy, h, rstd, w, dh_in = make_backward(M, N, dtype, F32 if through else dtype, through)
        dh, grad = o.room(M, N, dtype, pad=8), F32 if through else dtype
        dw = torch.randn((N,), device="cuda").to(grad)
        before = dw.clone() if through else None
        room = torch.full((M * N * 4,), 0xEE, dtype=torch.uint8, device="cuda")

        def call():
            backward(dy, h, rstd, w, dh_in, dh, dw, through, workspace=room)
        call()
        check_gradients(dy, h, rstd, w, dh_in, dh, dw, before)
        assert o.untouched(dh)
        # either alone, the same bits
        dh2, dw2 = o.room(M, N, dtype), before.clone() if through else torch.empty_like(dw)
        backward(dy, h, rstd, w, dh_in, dh2, None)
        assert torch.equal(bits(dh), bits(dh2))
        backward(dy, h, rstd, w, dh_in, o.room(M, N, dtype), dw2, through)
        assert torch.equal(dw, dw2)
        assert [k for _, k, _ in variants(call, "norm_backward_kernel")] == [
            (int(dtype is BF16), vpt, depth[0 if through else 1], int(through), whole)]


@pytest.mark.parametrize("N", [2048, 2043, 8192])
@pytest.mark.parametrize("over", ["dy", "h", "dh_in"])
def test_backward_in_place_with_rows_in_flight(N, over):
    M = 2500 if N < 8192 else 700
    dy, h, rstd, w, dh_in = make_backward(M, N, BF16, BF16, True)
    b = {"dy": dy.clone(), "h": h.clone(), "dh_in": dh_in.clone()}
    dh, dw = {"dy": dy, "h": h, "dh_in": dh_in}[over], torch.empty((N,), device="cuda")
    backward(dy, h, rstd, w, dh_in, dh, dw)
    check_gradients(b["dy"], b["h"], rstd, w, b["dh_in"], dh, dw)


@pytest.mark.parametrize("M,N", [(2500, 2048), (2500, 2043), (700, 8192)])
def test_backward_with_rows_in_flight_in_a_graph(M, N):
    dy, h, rstd, w, dh_in = make_backward(M, N, F16, F16, True)
    dh, dw = o.room(M, N, F16), torch.empty((N,), device="cuda")
    room = torch.empty((M * N * 4,), dtype=torch.uint8, device="cuda")
    backward(dy, h, rstd, w, dh_in, dh, dw, workspace=room)
    want = dh.clone(), dw.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        backward(dy, h, rstd, w, dh_in, dh, dw, workspace=room)
    for _ in range(3):
        dh.zero_(), dw.zero_(), room.fill_(0xFF)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(want[0], dh) and torch.equal(want[1], dw)


def test_backward_of_rows_that_are_not_ordinary_with_rows_in_flight():
    """NaN and infinities stay in their rows, whatever rows are copied beside them."""
    M, N = 2500, 2043
    dy, h, rstd, w, dh_in = make_backward(M, N, BF16, BF16, True)
    dy[7, 5], h[900, 2042], dh_in[2499, 0], rstd[1300] = float("nan"), float("inf"), float("inf"), 0.0
    dh, dw = o.room(M, N, BF16), torch.empty((N,), device="cuda")
    backward(dy, h, rstd, w, dh_in, dh, dw)
    bad = ~dh.isfinite().all(1)
    assert bad.nonzero()[:, 0].tolist() == [7, 900, 2499] and (~dh[2499].isfinite()).sum() == 1
    assert torch.equal(dh[1300], dh_in[1300])
    assert (~dw.isfinite()).nonzero()[:, 0].tolist() == [5, 2042]
    keep = [k for k in range(M) if k not in (7, 900, 2499)]
    want, size, _, _ = gradients64(dy, h, rstd, w, dh_in)
    tol = size * (N / 512 + 52) * 2.0 ** -24 + o.half_ulp(want, BF16) * 1.01
    assert ((dh.double() - want).abs() <= tol)[keep].all()


@pytest.mark.parametrize("pad", [0, 1])
def test_forward_of_the_smallest_rows(pad):
    """Squares are summed in float32: with eps 0, rows down to 1e-19 are normed like others, and rows whose squares
    all vanish have an infinite rstd; an eps covers them."""
    N = 700
    x, _, w = make(6, N, BF16, residual=False, pad=pad)
    x[0] *= 2.0 ** -60
    x[1:3] *= 2.0 ** -90
    x[3] *= 2.0 ** -120
    x[4, 1:] = 0
    for eps in (0.0, 1e-6):
        y, rstd = o.room(6, N, BF16, pad), torch.empty((6,), device="cuda")
        norm(x, None, w, eps=eps, y=y, rstd=rstd)
        if eps == 0:
            check_norm(x[[0, 4, 5]], None, w, eps, None, y[[0, 4, 5]], None, None, rstd[[0, 4, 5]])
            assert (rstd[1:4] == float("inf")).all()
            assert (y[1:4].isinf() | (x[1:4] == 0)).all()
        else:
            assert ((rstd[:4] - 1000).abs() < 1e-2).all()
            check_norm(x[[0, 1, 2, 4, 5]], None, w, eps, None, y[[0, 1, 2, 4, 5]], None, None, rstd[[0, 1, 2, 4, 5]])


@pytest.mark.parametrize("M,N,calls", [(2500, 8192, 1), (3000, 2048, 1), (4000, 700, 1), (150, 8192, 6)])
@pytest.mark.parametrize("pad", [0, 1])
def test_rstd_is_that_of_an_exact_sum(M, N, calls, pad):
    """rstd's last bit decides thousands of elements of y.  The kernels' orders of additions, gone through on the CPU,
    give the rstd of an exact sum (divided, eps added, root, reciprocal, each rounded once) for 0.905 to 0.94 of the
    bfloat16 rows, the same with plain sums for 0.66 to 0.856; 900 rows and more leave at most 0.008 of either to chance."""
    equal = 0
    for seed in range(calls):
        x, _, w = make(M, N, BF16, seed=seed, residual=False, pad=pad)
        rstd = torch.empty((M,), device="cuda")
        norm(x, None, w, y=o.room(M, N, BF16), rstd=rstd)
        total = x.double().square().sum(1).float().cpu().numpy()
        f = np.float32
        equal += int((rstd.cpu().numpy() == f(1) / np.sqrt(total / f(N) + f(1e-6))).sum())
    assert equal >= 0.88 * M * calls
