"""How much scratch memory the operators ask for, and that they use no more (no GPU needed: the checks)."""
import pytest

import gemm_gather_gb300 as gg
from tests.test_block_ops_host import BF16, F16, F32, INVALID, at, packed, refused

WHOLE = gg.linear_backward8_workspace(100, 500)


@pytest.mark.parametrize("kw", [dict(gdt=BF16, act=a) for a in ("none", "relu", "gelu", "gelu_tanh", "silu")]
                         + [dict(gdt=F32, act=a) for a in ("none", "relu")] + [dict(dtype=F16, gdt=F16, act="silu")])
def test_one_part_of_x_is_enough(kw):
    packed(ws_bytes=WHOLE // 2, **kw)
    refused(INVALID, packed, ws_bytes=WHOLE // 2 - 1, **kw)
    # an output may begin where the half ends
    packed(ws_bytes=WHOLE // 2, db=at(7) + WHOLE // 2, **kw)
    refused(INVALID, packed, ws_bytes=WHOLE // 2, db=at(7) + WHOLE // 2 - 4, **kw)


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
def test_two_parts_where_float32_gradients_need_them(act):
    packed(act=act, gdt=F32, ws_bytes=WHOLE)
    refused(INVALID, packed, act=act, gdt=F32, ws_bytes=WHOLE - 1)
    packed(act=act, gdt=F32, db=at(7) + WHOLE)
    refused(INVALID, packed, act=act, gdt=F32, db=at(7) + WHOLE - 4)
