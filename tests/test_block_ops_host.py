"""Host-side tests of the norm's and the 8-bit activations' C ABI (no GPU needed): what the checks
accept, every documented refusal, and what the binding looks at in a tensor.  Addresses are never
dereferenced."""
import pytest
import torch

import gemm_gather_gb300 as gg
from gemm_gather_gb300 import _lib

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
A = 1 << 36
STEP = 1 << 30
INVALID, ALIGN, UNSUP = _lib.GG_ERR_INVALID_ARG, _lib.GG_ERR_ALIGNMENT, _lib.GG_ERR_UNSUPPORTED


def at(i):
    return A + i * STEP


def refused(status, call, *args, **kw):
    with pytest.raises(gg.GGError) as e:
        call(*args, **kw)
    assert e.value.status == status, str(e.value)


def norm(**kw):
    a = dict(x=at(0), ldx=200, r=at(1), ldr=208, w=at(2), eps=1e-6, h=at(3), ldh=200, y=at(4), ldy=200, codes=at(5),
             ldc=208, scales=at(6), lds=2, rstd=at(7), M=100, N=200, dtype=BF16, weight_dtype=None)
    a.update(kw)
    gg.rms_norm_check(*list(a.values())[:-1], weight_dtype=a["weight_dtype"])


def test_norm_accepts():
    norm()
    norm(r=None, h=None, rstd=None, ldr=0, ldh=0)
    norm(y=None, ldy=0)
    norm(codes=None, scales=None, ldc=0, lds=0)
    norm(h=at(0)), norm(h=at(1), ldh=208), norm(y=at(0)), norm(h=at(1), ldh=208, y=at(0))
    norm(w=at(2) + 4, weight_dtype=F32), norm(w=at(2) + 2)
    norm(x=at(0) + 2, ldx=201, codes=at(5) + 1, ldc=201)
    norm(M=0, x=None, w=None, y=None), norm(N=0, x=None, w=None)
    norm(x=at(0), ldx=1000, h=at(0) + 400, ldh=1000)      # column ranges of one buffer


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=F32), UNSUP), (dict(weight_dtype=F16), UNSUP), (dict(M=-1), INVALID), (dict(N=1 << 31), UNSUP),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(y=None, codes=None, scales=None), INVALID),
    (dict(scales=None), INVALID), (dict(codes=None), INVALID), (dict(ldx=199), INVALID), (dict(ldr=1), INVALID),
    (dict(ldc=199), INVALID), (dict(lds=1), INVALID), (dict(ldh=0), INVALID), (dict(ldy=5), INVALID),
    (dict(x=at(0) + 1), ALIGN), (dict(w=at(2) + 2, weight_dtype=F32), ALIGN), (dict(rstd=at(7) + 2), ALIGN),
    (dict(scales=at(6) + 2), ALIGN), (dict(h=at(0), ldh=208), INVALID), (dict(y=at(3)), INVALID),
    (dict(h=at(0), y=at(0)), INVALID), (dict(codes=at(0)), INVALID), (dict(scales=at(5) + 64), INVALID),
    (dict(rstd=at(0)), INVALID), (dict(y=at(2)), INVALID), (dict(rstd=at(6)), INVALID), (dict(ldx=1 << 58), UNSUP)])
def test_norm_refuses(kw, status):
    refused(status, norm, **kw)


def backward(**kw):
    a = dict(dy=at(0), lddy=200, h=at(1), ldh=208, rstd=at(2), w=at(3), dh_in=at(4), lddhin=200, dh=at(5), lddh=200,
             dw=at(6), gdt=F32, acc=False, ws=at(7), M=100, N=200, dtype=BF16, weight_dtype=None,
             ws_bytes=gg.rms_norm_backward_workspace(100, 200))
    a.update(kw)
    gg.rms_norm_backward_check(*list(a.values())[:-2], weight_dtype=a["weight_dtype"], workspace_bytes=a["ws_bytes"])


def test_norm_backward_accepts():
    backward()
    backward(dw=None, ws=None, ws_bytes=0), backward(dh=None, dh_in=None)
    backward(dh=at(0)), backward(dh=at(1), lddh=208), backward(dh=at(4))
    backward(gdt=BF16, dw=at(6) + 2), backward(weight_dtype=F32), backward(dh_in=None, lddhin=0)
    backward(M=0, dy=None, h=None, rstd=None, w=None, ws=None, ws_bytes=0, dh=None)
    backward(dh=None, dh_in=at(6))                        # not read, so it may lie anywhere
    assert gg.rms_norm_backward_workspace(100, 200) == 100 * 200 * 4
    assert gg.rms_norm_backward_workspace(1 << 20, 10) == 608 * 10 * 4
    assert gg.rms_norm_backward_workspace(0, 5) == gg.rms_norm_backward_workspace(-3, 5) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=F32), UNSUP), (dict(gdt=F16), UNSUP), (dict(weight_dtype=F16), UNSUP), (dict(N=-1), INVALID),
    (dict(dy=None), INVALID), (dict(h=None), INVALID), (dict(rstd=None), INVALID), (dict(w=None), INVALID),
    (dict(ws=None), INVALID), (dict(ws_bytes=79999), INVALID), (dict(ws=at(7) + 2), ALIGN), (dict(lddy=199), INVALID),
    (dict(lddh=0), INVALID), (dict(dh=at(0), lddh=208), INVALID), (dict(dh=at(3)), INVALID), (dict(dw=at(5)), INVALID),
    (dict(dw=at(0)), INVALID), (dict(ws=at(0)), INVALID), (dict(ws=at(5)), INVALID), (dict(ws=at(6)), INVALID),
    (dict(dw=at(6) + 2), ALIGN), (dict(dh=at(5) + 1), ALIGN), (dict(dw=at(2)), INVALID), (dict(lddhin=3), INVALID)])
def test_norm_backward_refuses(kw, status):
    refused(status, backward, **kw)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), INVALID), (dict(codes=None), INVALID), (dict(scales=None), INVALID), (dict(dtype=F32), UNSUP),
    (dict(M=-1), INVALID), (dict(ldx=199), INVALID), (dict(ldc=3), INVALID), (dict(lds=1), INVALID),
    (dict(x=at(0) + 1), ALIGN), (dict(scales=at(2) + 1), ALIGN), (dict(codes=at(0)), INVALID), (dict(scales=at(0)), INVALID),
    (dict(scales=at(1)), INVALID)])
def test_pack_and_unpack_refuse(kw, status):
    a = dict(x=at(0), ldx=200, codes=at(1), ldc=200, scales=at(2), lds=2, M=100, N=200, dtype=F16)
    a.update(kw)
    v = list(a.values())
    refused(status, gg.pack8, *v, stream=0)
    if "scales" in kw and kw["scales"] == at(1):
        return                                            # inputs may overlap each other
    refused(status, gg.unpack8, *v[2:6], "silu", *v[:2], *v[6:], stream=0)


def test_unknown_activation():
    assert gg.lib.gg_unpack8(at(0), 128, at(1), 1, 7, at(2), 128, 4, 128, 0, None) == INVALID


def packed(**kw):
    a = dict(dZ=at(0), lddz=200, codes=at(1), ldc=512, scales=at(2), lds=4, act="silu", W=at(3), ldw=200, layout="kn",
             dX=at(4), lddx=500, dW=at(5), lddw=200, db=at(6), gdt=F32, acc=False, ws=at(7), M=100, N=200, K=500,
             dtype=BF16, path="auto", ws_bytes=gg.linear_backward8_workspace(100, 500))
    a.update(kw)
    return gg.linear_backward8_check(*list(a.values())[:-2], path=a["path"], workspace_bytes=a["ws_bytes"])


def test_linear_backward8_accepts():
    assert gg.linear_backward8_workspace(100, 500) == 2 * 100 * 504 * 2 and gg.linear_backward8_workspace(0, 5) == 0
    assert packed() == ("pair", "pair") and packed(path="split") == ("split", "split")
    assert packed(dX=None, W=None, path="split") == ("none", "split")
    assert packed(dW=None, ws=None, ws_bytes=0, path="pair") == ("pair", "none")
    assert packed(dW=None, ws=None, ws_bytes=0, act="none", codes=None, scales=None, path="pair") == ("pair", "none")
    assert packed(dW=None, dX=None, W=None, codes=None, scales=None, ws=None, ws_bytes=0) == ("none", "none")
    assert packed(codes=at(1) + 3, ldc=501, scales=at(2) + 4) == ("pair", "pair")
    assert packed(M=0, dZ=None, codes=None, scales=None, ws=None, ws_bytes=0) == ("none", "none")
    # the plan is linear_backward's
    for M, N, K in ((1, 64, 64), (777, 1000, 1523), (4096, 3584, 8192)):
        b = dict(M=M, N=N, K=K, lddz=N, ldc=K, lds=-(-K // 128), ldw=N, lddx=K, lddw=N, codes=at(40), dZ=at(60), W=at(80),
                 dX=at(100), dW=at(120), scales=at(140), ws=at(160), ws_bytes=gg.linear_backward8_workspace(M, K))
        assert packed(**b) == gg.linear_backward_check(at(60), N, at(160), -(-K // 8) * 8, at(80), N, "kn", at(40), K, "silu",
                                                       at(100), K, at(120), N, at(6), F32, False, M, N, K, BF16)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=F32), UNSUP), (dict(gdt=F16), UNSUP), (dict(K=-1), INVALID), (dict(dZ=None), INVALID), (dict(W=None), INVALID),
    (dict(codes=None), INVALID), (dict(scales=None), INVALID), (dict(ws=None), INVALID), (dict(ws_bytes=2 * 100 * 504 * 2 - 1), INVALID),
    (dict(ws=at(7) + 8), ALIGN), (dict(lddz=201), ALIGN), (dict(W=at(3) + 2), ALIGN), (dict(ldc=499), INVALID),
    (dict(lds=3), INVALID), (dict(scales=at(2) + 2), ALIGN), (dict(dX=at(1)), INVALID), (dict(dW=at(2)), INVALID),
    (dict(db=at(1) + 40), INVALID), (dict(ws=at(1)), INVALID), (dict(ws=at(2)), INVALID), (dict(ws=at(0)), INVALID),
    (dict(ws=at(3)), INVALID), (dict(ws=at(4)), INVALID), (dict(ws=at(5)), INVALID), (dict(ws=at(6)), INVALID),
    (dict(dX=at(0)), INVALID), (dict(M=1 << 31), UNSUP)])
def test_linear_backward8_refuses(kw, status):
    refused(status, packed, **kw)


def zeros(*shape, dtype=BF16):
    return torch.zeros(shape, dtype=dtype)


@pytest.mark.parametrize("kw,says", [
    (dict(x=zeros(100, 200, dtype=F16)), "x: a tensor of torch.bfloat16"), (dict(x=zeros(100, 200)), "x: a tensor on the GPU"),
    (dict(r=zeros(99, 200)), "residual: a tensor of 20000"), (dict(w=zeros(199)), "weight: a tensor of 200"),
    (dict(w=zeros(400)[::2]), "weight: a contiguous"), (dict(codes=zeros(100, 200, dtype=torch.int8)), "codes: a tensor of torch.uint8"),
    (dict(codes=zeros(100, 199, dtype=torch.uint8)), "codes: a tensor of 20000"),
    (dict(scales=zeros(100, 1, dtype=F32)), "scales: a tensor of 200"), (dict(rstd=zeros(100)), "rstd: a tensor of torch.float32"),
    (dict(y=zeros(100, 100)), "y: a tensor of 20000"), (dict(h=zeros(100, 200)), "h: a tensor on the GPU")])
def test_norm_looks_at_tensors(kw, says):
    with pytest.raises(ValueError, match=says):
        norm(**kw)


def test_the_others_look_at_tensors():
    for kw, says in ((dict(ws=zeros(100, 200)[:, :100]), "workspace: a contiguous"), (dict(ws=zeros(10)), "workspace: a tensor of 80000"),
                     (dict(dy=zeros(5)), "dy: a tensor of 20000"), (dict(dw=zeros(200)), "dweight: a tensor of torch.float32"),
                     (dict(ws=zeros(40000)), "workspace: a tensor on the GPU")):
        with pytest.raises(ValueError, match=says):
            backward(**kw)
    for kw, says in ((dict(codes=zeros(100, 500)), "codes: a tensor of torch.uint8"), (dict(scales=zeros(5, dtype=F32)), "scales: a tensor of 400"),
                     (dict(dZ=zeros(5)), "dZ: a tensor of 20000"), (dict(dW=zeros(500, 200)), "dW: a tensor of torch.float32")):
        with pytest.raises(ValueError, match=says):
            packed(**kw)
    with pytest.raises(ValueError, match="out: a tensor of torch.float16"):
        gg.unpack8(at(0), 128, at(1), 1, "none", zeros(4, 128), 128, 4, 128, F16, stream=0)


def entropy(**kw):
    a = dict(X=at(0), ldx=520, W=at(1), ldw=520, layout="nk", target=at(2), weight=at(3), stats=at(4), loss=at(5), lse=at(6),
             dX=at(7), lddx=513, dW=at(8), lddw=513, gdt=F32, acc=False, ws=at(9), T=100, V=5000, K=513, dtype=BF16, piece=0,
             grad_scale=1.0, ws_bytes=None)
    a.update(kw)
    if a["ws_bytes"] is None:
        a["ws_bytes"] = gg.linear_cross_entropy_workspace(a["T"], a["V"], a["K"], max(a["piece"], 0),
                                                          a["dX"] is not None or a["dW"] is not None)
    gg.linear_cross_entropy_check(*list(a.values())[:-3], piece=a["piece"], grad_scale=a["grad_scale"],
                                  workspace_bytes=a["ws_bytes"])


def test_entropy_accepts():
    entropy()
    entropy(layout="kn", ldw=5000, lddw=5000)
    entropy(dX=None, dW=None), entropy(dX=None), entropy(dW=None), entropy(stats=None, lse=None)
    entropy(dX=at(0), lddx=520)                           # dX over X
    entropy(gdt=BF16, dW=at(8) + 2), entropy(piece=128), entropy(piece=1 << 20)
    entropy(T=0, X=None, W=None, target=None, weight=None, loss=None, ws=None, ws_bytes=0)
    entropy(T=0, V=0, X=None, W=None, target=None, weight=None, loss=None, ws=None, ws_bytes=0)
    entropy(K=0, X=None, W=None)
    small = gg.linear_cross_entropy_workspace(4096, 100003, 2048, 0, False)
    assert 4096 * 2048 * 2 < small < 4096 * 100003 * 2 // 16
    assert gg.linear_cross_entropy_workspace(100, 5000, 513, 1024) < gg.linear_cross_entropy_workspace(100, 5000, 513)
    assert gg.linear_cross_entropy_workspace(0, 5, 5) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=F32), UNSUP), (dict(gdt=F16), UNSUP), (dict(T=-1), INVALID), (dict(V=0, W=None), INVALID), (dict(V=1 << 31), UNSUP),
    (dict(piece=100), INVALID), (dict(piece=-128), INVALID), (dict(grad_scale=float("nan")), INVALID),
    (dict(grad_scale=float("inf")), INVALID), (dict(X=None), INVALID), (dict(W=None), INVALID), (dict(target=None), INVALID),
    (dict(weight=None), INVALID), (dict(loss=None), INVALID), (dict(ws=None), INVALID), (dict(ws_bytes=1000), INVALID),
    (dict(ws=at(9) + 8), ALIGN), (dict(X=at(0) + 8), ALIGN), (dict(W=at(1) + 2), ALIGN), (dict(ldx=521), ALIGN),
    (dict(ldw=512), INVALID), (dict(ldw=525), ALIGN), (dict(target=at(2) + 4), ALIGN), (dict(weight=at(3) + 2), ALIGN),
    (dict(stats=at(4) + 1), ALIGN), (dict(dW=at(8) + 2), ALIGN), (dict(dX=at(0)), INVALID), (dict(dX=at(1)), INVALID),
    (dict(dW=at(1)), INVALID), (dict(loss=at(6)), INVALID), (dict(lse=at(3)), INVALID), (dict(stats=at(5)), INVALID),
    (dict(ws=at(0)), INVALID), (dict(ws=at(1)), INVALID), (dict(ws=at(7)), INVALID), (dict(ws=at(8)), INVALID),
    (dict(loss=at(9) + 64), INVALID), (dict(loss=at(2)), INVALID), (dict(lddx=512), INVALID), (dict(lddw=1), INVALID)])
def test_entropy_refuses(kw, status):
    refused(status, entropy, **kw)


@pytest.mark.parametrize("kw,says", [
    (dict(X=zeros(100, 513, dtype=F16)), "X: a tensor of torch.bfloat16"), (dict(W=zeros(100, 513)), "W: a tensor of 2565000"),
    (dict(target=zeros(100, dtype=torch.int32)), "target: a tensor of torch.int64"), (dict(weight=zeros(100)), "weight: a tensor of"),
    (dict(stats=zeros(1, dtype=F32)), "stats: a tensor of 2"), (dict(loss=zeros(99, dtype=F32)), "loss: a tensor of 100"),
    (dict(dW=zeros(5000, 513)), "dW: a tensor of torch.float32"), (dict(dX=zeros(100, 513)), "dX: a tensor on the GPU"),
    (dict(ws=zeros(1 << 10), ws_bytes=1 << 20), "workspace: a tensor of 1048576")])
def test_entropy_looks_at_tensors(kw, says):
    with pytest.raises(ValueError, match=says):
        entropy(**kw)
