"""What the operators' binding looks at in a tensor before it hands out its address: type, size and
device.  (No GPU needed: the device comes last, so tensors on the CPU show the other refusals.)"""
import pytest
import torch

import gemm_gather_gb300 as gg

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
A = 1 << 36


def linear(**kw):
    a = dict(X=A, ldx=24, W=A + (1 << 30), ldw=24, layout="nk", bias=None, act="none", residual=None, ldr=16,
             Y=A + (2 << 30), ldy=16, z=None, ldz=16, M=5, N=16, K=24, dtype=BF16, path="auto", bias_dtype=None)
    a.update(kw)
    return gg.linear_check(*a.values())


def zeros(*shape, dtype=BF16):
    return torch.zeros(shape, dtype=dtype)


@pytest.mark.parametrize("kw,says", [
    (dict(X=zeros(5, 24, dtype=F32)), "X: a tensor of torch.bfloat16"), (dict(X=zeros(4, 24)), "X: a tensor of 120 elements"),
    (dict(X=zeros(5, 24)), "X: a tensor on the GPU"), (dict(W=zeros(16, 23)), "W: a tensor of 384 elements"),
    (dict(X=zeros(5, 32)[:, 8:], ldx=32), "X: a tensor on the GPU"),      # a part of wider rows
    (dict(bias=zeros(15)), "bias: a tensor of 16 elements"), (dict(bias=zeros(32)[::2]), "bias: a contiguous tensor"),
    (dict(bias=zeros(16, dtype=F16), bias_dtype=F32), "bias: a tensor of torch.float32"),
    (dict(bias=zeros(16, dtype=F32)), "bias: a tensor on the GPU"),       # a float32 bias is one of the types
    (dict(residual=zeros(5, 15)), "residual: a tensor of 80"), (dict(Y=zeros(5, 16, dtype=F16)), "Y: a tensor of torch.bfl"),
    (dict(z=zeros(79)), "z: a tensor of 80"), (dict(z=zeros(80)), "z: a tensor on the GPU")])
def test_linear(kw, says):
    with pytest.raises(ValueError, match=says):
        linear(**kw)


def test_what_is_not_read_may_be_anything():
    assert linear(M=0, X=None, W=None) == "none"
    with pytest.raises(ValueError, match="X: a tensor on the GPU"):
        linear(M=0, X=zeros(1))                                           # no size is asked of it
    b = dict(dZ=A, lddz=16, X=A + (1 << 30), ldx=24, W=zeros(1, dtype=F32), ldw=24, layout="nk", z_in=zeros(1), ldzin=24,
             act="silu", dX=None, lddx=24, dW=A + (2 << 30), lddw=24, db=None, gdt=F32, acc=False, M=5, N=16, K=24,
             dtype=BF16)
    assert gg.linear_backward_check(*b.values())[0] == "none"
    b.update(dX=A + (3 << 30))
    with pytest.raises(ValueError, match="W: a tensor of torch.bfloat16"):
        gg.linear_backward_check(*b.values())
    b.update(W=A + (4 << 30), dW=zeros(16, 24))
    with pytest.raises(ValueError, match="z_in: a tensor of 120"):
        gg.linear_backward_check(*b.values())
    b.update(z_in=None)
    with pytest.raises(ValueError, match="dW: a tensor of torch.float32"):
        gg.linear_backward_check(*b.values())


@pytest.mark.parametrize("kw,says", [
    (dict(target=zeros(6, dtype=torch.int32)), "target: a tensor of torch.int64"),
    (dict(target=zeros(5, dtype=torch.int64)), "target: a tensor of 6"),
    (dict(weight=torch.tensor(1.0).expand(6)), "weight: a contiguous tensor"),
    (dict(advantage=zeros(6, dtype=torch.float64)), "advantage: a tensor of torch.float32"),
    (dict(old_logp=zeros(6, dtype=BF16)), "old_logp: a tensor of"), (dict(stats=zeros(3, dtype=F32)), "stats: a tensor of 4"),
    (dict(logits=zeros(6, 99)), "logits: a tensor of 600"), (dict(dlogits=zeros(6, 100, dtype=F32)), "dlogits: a tensor of"),
    (dict(logp_out=zeros(6, dtype=F32)), "logp_out: a tensor on the GPU")])
def test_policy_loss(kw, says):
    a = dict(logits=A, ld=100, target=A + (1 << 30), old_logp=None, ref_logp=None, advantage=A + (2 << 30),
             weight=A + (3 << 30), T=6, V=100, dtype=BF16, stats=None, logp_out=A + (4 << 30), dlogits=None, ldd=100)
    gg.policy_loss_check(*a.values())
    a.update(kw)
    with pytest.raises(ValueError, match=says):
        gg.policy_loss_check(*a.values())


def test_adamw():
    t = dict(param=torch.zeros(300), grad=torch.zeros(300), m=torch.zeros(300), v=torch.zeros(300))
    with pytest.raises(ValueError, match="param of tensor 0: a tensor on the GPU"):
        gg.adamw_check(gg.adamw_tensors([t]), 1, 1e-3)
    for bad, bits in ((dict(m=zeros(300, dtype=torch.int32)), 32), (dict(param=zeros(300, dtype=torch.float64)), 32),
                      (dict(m=zeros(300, dtype=torch.int8), v=zeros(300, dtype=torch.uint8)), 8)):
        with pytest.raises(ValueError, match="does not do"):
            gg.adamw_tensors([{**t, **bad}], state_bits=bits)
    with pytest.raises(ValueError, match="grad_scale: a tensor of torch.float32"):
        gg.adamw_check(gg.adamw_tensors([]), 1, 1e-3, grad_scale=zeros(1, dtype=torch.float64))


@pytest.mark.parametrize("M", [1, 16, 27, 100, 300, 777, 2048])
def test_the_kernel_does_not_depend_on_addresses(M):
    """Where operands lie may not change the order of their sums."""
    for N in (512, 1024, 3584, 8192):
        for K in (512, 1000, 2048, 4096):
            def chosen(shift):
                a = dict(X=A + shift, ldx=K, W=A + (1 << 34) + shift, ldw=K, layout="nk", bias=None, act="none",
                         residual=None, ldr=N, Y=A + (2 << 34), ldy=N, z=None, ldz=N, M=M, N=N, K=K, dtype=BF16)
                b = dict(dZ=A + shift, lddz=N, X=A + (1 << 34) + shift, ldx=K, W=A + (2 << 34) + shift, ldw=K,
                         layout="nk", z_in=None, ldzin=K, act="none", dX=A + (3 << 34), lddx=K, dW=A + (4 << 34), lddw=K,
                         db=None, gdt=F32, acc=False, M=M, N=N, K=K, dtype=BF16)
                return gg.linear_check(*a.values()), gg.linear_backward_check(*b.values())
            assert chosen(0) == chosen(16) == chosen(112)


def test_pitches_that_a_tensor_map_does_not_hold():
    """A single row may have any pitch as far as memory goes; the check refuses what the launch would."""
    from gemm_gather_gb300 import _lib
    limit = 1 << 39
    assert linear(M=1, ldx=limit - 8) == "split"
    assert linear(M=1, ldy=limit, residual=A + (3 << 30), ldr=limit) == "split"
    for kw in (dict(M=1, ldx=limit), dict(N=1, ldw=limit)):
        with pytest.raises(gg.GGError) as e:
            linear(**kw)
        assert e.value.status == _lib.GG_ERR_UNSUPPORTED
