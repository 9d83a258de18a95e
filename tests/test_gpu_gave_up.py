"""Launches that gave up on a wait leave nothing behind: what they had on its way has landed before
they end, and a launch right behind them, on the same SMs, is right."""
import time

import pytest
import torch

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
