"""Equal inputs give equal bits wherever they lie in memory (the linear layer: test_gpu_linear_edges.py)."""
import pytest
import torch

import gg_inputs
from tests.test_gpu_adamw import BF16, F16, F32, make, run
from tests.test_gpu_policy_loss import call
from tests.test_gpu_policy_loss import make as make_loss

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("T,V,offset", [(5, 12345, 0), (40, 20011, 1), (3, 100003, 3), (300, 1000, 0), (2, 500001, 1)])
def test_policy_loss_at_the_same_offset_from_a_16_byte_boundary(T, V, offset, dtype):
    """Rows at the same places between 16-byte boundaries, the whole at other addresses."""
    vec = 4 if dtype == F32 else 8
    c = make_loss(T, V, dtype, shift=offset, masked=0.2, seed=V)
    want = call(c)
    base = c["logits"]
    for steps in (1, 5, 8):
        buf = torch.empty(T * V + offset + 8 * vec, dtype=dtype, device="cuda")
        first = offset + steps * vec
        c["logits"] = buf[first:first + T * V].view(T, V).copy_(base)
        got = call(c, gshift=steps)                 # the gradient's own place does not matter
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("param,grad,copy", [(F32, BF16, BF16), (BF16, F32, None), (F16, F16, None)])
def test_adamw_wherever_the_tensors_lie(param, grad, copy, bits):
    first = None
    for shift in (0, 8, 4, 1):
        t = make(70000, param, grad, bits, copy, shift, gen=gg_inputs.generator(5))
        run([t], 3, bits)
        got = [t[k].clone() for k in ("param", "m", "v", "m_scale", "v_scale", "copy") if t.get(k) is not None]
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(first, got))
