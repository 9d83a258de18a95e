"""The operators write nothing behind the scratch memory they ask for."""
import pytest
import torch

import gemm_gather_gb300 as gg
from tests import block_oracle as o
from tests.block_oracle import BF16, F32
from tests.test_gpu_pack8 import layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act,gdt", [("silu", BF16), ("gelu", BF16), ("none", F32), ("relu", F32)])
@pytest.mark.parametrize("path", ["split", "pair"])
def test_backward8_with_half_of_the_scratch_memory(act, gdt, path):
    M, N, K = 130, 264, 520
    codes, scales, w, dz = layer(M, N, K, BF16, "nk")
    whole = gg.linear_backward8_workspace(M, K)
    got = []
    for n in (whole, whole // 2):
        room = torch.full((whole + 64,), 0xEE, dtype=torch.uint8, device="cuda")
        dx, dw = o.room(M, K, BF16), torch.empty(w.shape, device="cuda").to(gdt)
        gg.linear_backward8(dz, dz.stride(0), codes, codes.stride(0), scales, scales.stride(0), act, w, w.stride(0), "nk",
                            dx, dx.stride(0), dw, dw.stride(0), None, gdt, False, room, M, N, K, BF16, path=path,
                            workspace_bytes=n)
        assert (room[n:] == 0xEE).all()
        got.append((dx.clone(), dw))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
