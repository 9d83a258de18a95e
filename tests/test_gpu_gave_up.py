"""Launches that gave up on a wait leave nothing behind: what they had on its way has landed before
they end, and a launch right behind them, on the same SMs, is right."""
import time

import pytest
import torch

import gg_inputs
from tests import test_gpu_linear as lin
from tests.test_gpu_policy_loss import BF16, call, check, far_from_clip, make

pytestmark = pytest.mark.gpu


@pytest.fixture
def stall():
    """Launches between its two calls miss one message or one load; 2 ms of patience."""
    import gemm_gather_gb300 as gg
    old = gg.get_wait_limit_ns()

    def on(yes):
        gg.set_wait_limit_ns(2_000_000 if yes else old)
        gg.debug_inject_stall(yes)

    yield on
    on(False)


@pytest.mark.parametrize("T,V", [(1, 8192), (150, 100003), (300, 20011)])
def test_policy_loss_behind_one_that_gave_up(T, V, stall):
    c = far_from_clip(make(T, V, BF16, masked=0.0, seed=12))
    bad, good = (torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(2))
    torch.cuda.synchronize()
    begin = time.perf_counter()
    for _ in range(2):
        stall(True)
        call(c, status=bad)
        stall(False)
        got = call(c, status=good)
    torch.cuda.synchronize()
    assert time.perf_counter() - begin < 10       # 2 ms, then at most a second for what is late, each
    assert int(bad.item()) == -6 and int(good.item()) == 0
    check(c, got)


@pytest.mark.parametrize("path", ["split", "pair"])
@pytest.mark.parametrize("M,N,K", [(300, 300, 1024), (40, 260, 4096), (1100, 2000, 136)])
def test_linear_behind_one_that_gave_up(M, N, K, path, stall):
    gen = gg_inputs.generator(M)
    x, w = lin.mat(M, K, BF16, gen, ints=True), lin.mat(N, K, BF16, gen, ints=True)
    y, y2, dx = lin.out_mat(M, N, BF16), lin.out_mat(M, N, BF16), lin.out_mat(M, K, BF16)
    dw = torch.empty((N, K), device="cuda")
    dz = lin.mat(M, N, BF16, gen, ints=True)
    bad, good = (torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(2))
    torch.cuda.synchronize()
    begin = time.perf_counter()
    stall(True)
    lin.call_linear(x, w, "nk", None, "none", None, y, None, path, status=bad)
    lin.call_backward(dz, x, w, "nk", None, "none", dx, dw, None, False, path, status=bad)
    stall(False)
    lin.call_linear(x, w, "nk", None, "none", None, y2, None, path, status=good)
    lin.call_backward(dz, x, w, "nk", None, "none", dx, dw, None, False, path, status=good)
    torch.cuda.synchronize()
    assert time.perf_counter() - begin < 20
    assert int(bad.item()) == -6 and int(good.item()) == 0
    assert torch.equal(y2, (x.double() @ w.double().t()).to(BF16))
    assert torch.equal(dx, (dz.double() @ w.double()).to(BF16))
    assert torch.equal(dw.double(), dz.double().t() @ x.double())
