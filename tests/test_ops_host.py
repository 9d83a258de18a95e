"""Host-side tests of the operators' C ABI (no GPU needed): what the checks accept, which
kernel a product would run, and every documented refusal.  Addresses are never dereferenced."""
import random

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


def linear(**kw):
    a = dict(X=at(0), ldx=512, W=at(1), ldw=256, layout="kn", bias=at(2), act="gelu", residual=at(3), ldr=200,
             Y=at(4), ldy=200, z=at(5), ldz=200, M=100, N=200, K=500, dtype=F16, path="auto", bias_dtype=None)
    a.update(kw)
    return gg.linear_check(*[a[k] for k in ("X", "ldx", "W", "ldw", "layout", "bias", "act", "residual", "ldr", "Y",
                                            "ldy", "z", "ldz", "M", "N", "K", "dtype", "path", "bias_dtype")])


def test_linear_accepts():
    assert linear() == "split"
    assert linear(M=4096, N=4096, ldw=4096, ldr=4096, ldy=4096, ldz=4096) == "pair"
    assert linear(path="pair") == "pair" and linear(path="split") == "split"
    assert linear(layout="nk", ldw=504) == "split"
    assert linear(bias=None, residual=None, z=None, ldr=0, ldz=0) == "split"
    assert linear(residual=at(4)) == "split"              # the residual is Y itself
    assert linear(bias=at(2) + 4, bias_dtype=F32) == "split"
    assert linear(Y=at(4) + 2, ldy=201, residual=at(3) + 2, ldr=203) == "split"  # any alignment
    assert linear(M=0) == "none" and linear(N=0) == "none"
    assert linear(K=0, X=None, W=None, ldx=0) == "none"
    # Y and X as column ranges of one buffer of one pitch
    assert linear(X=at(0), ldx=1000, Y=at(0) + 1000, ldy=1000) == "split"


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=F32), UNSUP), (dict(M=-1), INVALID), (dict(K=-5), INVALID), (dict(M=1 << 31), UNSUP),
    (dict(X=None), INVALID), (dict(W=None), INVALID), (dict(Y=None), INVALID),
    (dict(ldx=496), INVALID), (dict(ldw=192), INVALID), (dict(ldy=199), INVALID), (dict(ldr=1), INVALID),
    (dict(ldz=0), INVALID), (dict(ldx=511), ALIGN), (dict(ldw=255), ALIGN), (dict(X=at(0) + 8), ALIGN),
    (dict(W=at(1) + 2), ALIGN), (dict(Y=at(4) + 1), ALIGN), (dict(bias=at(2) + 1), ALIGN),
    (dict(bias=at(2) + 2, bias_dtype=F32), ALIGN), (dict(bias_dtype=BF16), UNSUP),
    (dict(Y=at(0)), INVALID), (dict(Y=at(1) + 64), INVALID), (dict(z=at(4)), INVALID), (dict(z=at(3)), INVALID),
    (dict(residual=at(4) + 2), INVALID), (dict(residual=at(4), ldr=208), INVALID), (dict(bias=at(4)), INVALID),
    (dict(X=at(0), ldx=1000, Y=at(0) + 990, ldy=1000), INVALID),
    (dict(X=at(0), ldx=1000, Y=at(0) + 1800, ldy=1000), INVALID),   # its rows run into X's next row
    (dict(ldx=1 << 60), UNSUP),
])
def test_linear_refuses(kw, status):
    with pytest.raises(gg.GGError) as e:
        linear(**kw)
    assert e.value.status == status, str(e.value)


def test_unknown_codes_are_refused():
    ok = [at(0), 512, at(1), 256, 0, None, 0, 0, None, 0, at(4), 200, None, 0, 100, 200, 500, 0, 0, None]
    assert gg.lib.gg_linear_check(*ok) == 0
    for place, bad in ((4, 2), (7, 9), (7, -1), (18, 3), (17, 7)):
        args = list(ok)
        args[place] = bad
        assert gg.lib.gg_linear_check(*args) in (INVALID, UNSUP)
        assert gg.lib.gg_last_error()


def backward(**kw):
    a = dict(dZ=at(0), lddz=200, X=at(1), ldx=512, W=at(2), ldw=200, layout="kn", z_in=at(3), ldzin=500, act="silu",
             dX=at(4), lddx=500, dW=at(5), lddw=200, db=at(6), gdt=F32, acc=False, M=100, N=200, K=500, dtype=BF16,
             path="auto")
    a.update(kw)
    return gg.linear_backward_check(*[a[k] for k in ("dZ", "lddz", "X", "ldx", "W", "ldw", "layout", "z_in", "ldzin",
                                                     "act", "dX", "lddx", "dW", "lddw", "db", "gdt", "acc", "M", "N",
                                                     "K", "dtype", "path")])


def test_backward_accepts():
    assert backward() == ("pair", "pair")                  # both in one walk of the pairs
    assert backward(path="pair") == ("pair", "pair")
    assert backward(path="split") == ("split", "split")
    assert backward(dX=None, W=None, path="split") == ("none", "split")
    assert backward(dW=None, X=None, path="pair") == ("pair", "none")
    assert backward(dX=None, W=None) in (("none", "split"), ("none", "pair"))  # whichever is estimated faster
    assert backward(dW=None, X=None) in (("split", "none"), ("pair", "none"))
    assert backward(dW=None, dX=None, X=None, W=None) == ("none", "none")
    for path in ("auto", "split"):
        want = (("pair", "pair"), ("split", "split"))[path == "split"]
        assert backward(dX=at(3), path=path) == want       # dX over z_in
        assert backward(layout="nk", ldw=504, lddw=501, dW=at(5) + 4, path=path) == want
        assert backward(gdt=BF16, db=at(6) + 2, path=path) == want
    assert backward(M=0, dZ=None, X=None) == ("none", "none")


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=F32), UNSUP), (dict(gdt=F16), UNSUP), (dict(N=-1), INVALID), (dict(dZ=None), INVALID),
    (dict(X=None), INVALID), (dict(W=None), INVALID), (dict(lddz=203), ALIGN), (dict(lddz=192), INVALID),
    (dict(X=at(1) + 2), ALIGN), (dict(ldw=201), ALIGN), (dict(lddw=199), INVALID), (dict(lddx=8), INVALID),
    (dict(dW=at(5) + 2), ALIGN), (dict(dX=at(0)), INVALID), (dict(dX=at(1)), INVALID), (dict(dW=at(2)), INVALID),
    (dict(db=at(5)), INVALID), (dict(dX=at(3), lddx=504), INVALID), (dict(dW=at(4)), INVALID), (dict(db=at(0)), INVALID),
])
def test_backward_refuses(kw, status):
    with pytest.raises(gg.GGError) as e:
        backward(**kw)
    assert e.value.status == status, str(e.value)


@pytest.mark.parametrize("kw,status", [
    (dict(dy=None), INVALID), (dict(ld=9), INVALID), (dict(dtype=F32), UNSUP), (dict(dz=at(0) + 2), INVALID),
    (dict(z=at(1) + 1), ALIGN), (dict(M=-1), INVALID)])
def test_act_backward_refuses(kw, status):
    a = dict(dy=at(0), ld=10, z=at(1), dz=at(2), M=10, N=10, dtype=F16)
    a.update(kw)
    with pytest.raises(gg.GGError) as e:
        gg.act_backward(a["dy"], a["ld"], a["z"], 10, a["dz"], 10, "relu", a["M"], a["N"], a["dtype"], stream=0)
    assert e.value.status == status


def loss(**kw):
    a = dict(logits=at(0), ld=1000, target=at(1), old=at(2), ref=at(3), adv=at(4), weight=at(5), T=50, V=1000,
             dtype=BF16, stats=at(6), logp=at(7), dlogits=at(8), ldd=1000)
    opt = {k: kw.pop(k) for k in list(kw) if k in ("inv_temperature", "clip_low", "clip_high", "kl_coef", "grad_scale")}
    a.update(kw)
    gg.policy_loss_check(*[a[k] for k in ("logits", "ld", "target", "old", "ref", "adv", "weight", "T", "V", "dtype",
                                          "stats", "logp", "dlogits", "ldd")], **opt)


def test_loss_accepts():
    loss()
    loss(dlogits=at(0))
    loss(dlogits=None, stats=None, old=None, ref=None)
    loss(logits=at(0) + 2, ld=1001, dtype=F16)
    loss(T=0, logits=None, target=None, adv=None, weight=None, logp=None)


@pytest.mark.parametrize("kw,status", [
    (dict(logits=None), INVALID), (dict(target=None), INVALID), (dict(adv=None), INVALID), (dict(weight=None), INVALID),
    (dict(logp=None), INVALID), (dict(T=-1), INVALID), (dict(V=0), INVALID), (dict(ld=999), INVALID),
    (dict(ldd=999), INVALID), (dict(T=1 << 29), UNSUP), (dict(target=at(1) + 4), ALIGN), (dict(adv=at(4) + 2), ALIGN),
    (dict(logits=at(0) + 1), ALIGN), (dict(inv_temperature=0.0), INVALID), (dict(inv_temperature=float("nan")), INVALID),
    (dict(clip_low=-0.1), INVALID), (dict(clip_high=float("nan")), INVALID), (dict(kl_coef=float("inf")), INVALID),
    (dict(grad_scale=float("inf")), INVALID), (dict(dlogits=at(0) + 2), INVALID), (dict(dlogits=at(0), ldd=1008), INVALID),
    (dict(logp=at(2)), INVALID), (dict(stats=at(7)), INVALID), (dict(stats=at(0) + 400), INVALID), (dict(dtype=3), INVALID),
])
def test_loss_refuses(kw, status):
    with pytest.raises(gg.GGError) as e:
        loss(**kw)
    assert e.value.status == status, str(e.value)


def tensor(**kw):
    array = (gg.AdamwTensor * 1)()
    a = dict(param=at(0), grad=at(1), m=at(2), v=at(3), m_scale=at(4), v_scale=at(5), copy=at(6), n=1000,
             param_dtype=_lib.GG_F32, grad_dtype=_lib.GG_BF16, copy_dtype=_lib.GG_BF16, state_bits=8)
    a.update(kw)
    for k, x in a.items():
        setattr(array[0], k, x)
    return gg.AdamwTensors(array, [])


def test_adamw_accepts():
    gg.adamw_check(tensor(), 1, 1e-3)
    gg.adamw_check(tensor(state_bits=32, m_scale=None, v_scale=None, copy=None), 10 ** 7, 0.0, 0.0, 0.0, 0.0)
    gg.adamw_check(tensor(m=at(2) + 1, v=at(3) + 3, grad=at(1) + 2, param=at(0) + 4), 1, 1e-3)
    gg.adamw_check(tensor(n=0, param=None, grad=None, m=None, v=None), 1, 1e-3)
    gg.adamw_check(gg.adamw_tensors([]), 1, 1e-3)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), INVALID), (dict(param=None), INVALID), (dict(grad=None), INVALID), (dict(m=None), INVALID),
    (dict(v_scale=None), INVALID), (dict(state_bits=4), UNSUP), (dict(param_dtype=3), INVALID),
    (dict(grad_dtype=-1), INVALID), (dict(copy_dtype=_lib.GG_F32), UNSUP), (dict(param=at(0) + 2), ALIGN),
    (dict(state_bits=32, m=at(2) + 2), ALIGN), (dict(m_scale=at(4) + 1), ALIGN), (dict(v=at(2) + 999), INVALID),
    (dict(copy=at(0)), INVALID), (dict(grad=at(0) + 64), INVALID), (dict(n=1 << 41), UNSUP)])
def test_adamw_refuses_tensors(kw, status):
    with pytest.raises(gg.GGError) as e:
        gg.adamw_check(tensor(**kw), 1, 1e-3)
    assert e.value.status == status, str(e.value)


@pytest.mark.parametrize("args", [(0, 1e-3), (1, float("nan")), (1, 1e-3, 1.0), (1, 1e-3, -0.1), (1, 1e-3, 0.9, 1.0),
                                  (1, 1e-3, 0.9, 0.99, -1e-8), (1, 1e-3, 0.9, 0.99, float("inf")),
                                  (1, 1e-3, 0.9, 0.99, 1e-8, float("nan"))])
def test_adamw_refuses_settings(args):
    with pytest.raises(gg.GGError) as e:
        gg.adamw_check(tensor(), *args)
    assert e.value.status == INVALID


def test_adamw_tensors_checks_what_torch_knows():
    t = dict(param=torch.zeros(300), grad=torch.zeros(300), m=torch.zeros(300), v=torch.zeros(300))
    table = gg.adamw_tensors([t, t])
    assert table.count == 2 and table.array[1].n == 300 and table.array[0].state_bits == 32
    for bad in (dict(m=torch.zeros(299)), dict(grad=torch.zeros(300, 2)[:, 0]), dict(m=torch.zeros(300, dtype=F16))):
        with pytest.raises(ValueError):
            gg.adamw_tensors([{**t, **bad}])
    with pytest.raises(ValueError):
        gg.adamw_tensors([{**t, "m_scale": torch.zeros(1)}], state_bits=8)


@pytest.mark.parametrize("seed", range(3))
def test_linear_check_accepts_only_apart_buffers(seed):
    """Seeded random calls: an accepted one has 16-byte aligned operands whose pitches hold their
    rows, and no output element shares a byte with another argument (by enumeration of rows)."""
    rng = random.Random(seed)
    accepted = 0
    for _ in range(3000):
        M, N, K = rng.choice([1, 3, 8]), rng.choice([1, 8, 20]), rng.choice([0, 8, 24])
        pick = lambda: A + 2 * rng.choice([0, 8, 16, 64, 100, 400, 1000, 3000, 5000])  # noqa: E731
        ld = lambda: rng.choice([8, 16, 24, 40, 21])  # noqa: E731
        a = dict(X=pick(), ldx=ld(), W=pick() + 20000, ldw=ld(), layout=rng.choice(["kn", "nk"]), bias=None, act="none",
                 residual=rng.choice([None, pick()]), ldr=ld(), Y=pick(), ldy=ld(), z=rng.choice([None, pick()]), ldz=ld(),
                 M=M, N=N, K=K)
        try:
            linear(**a)
        except gg.GGError as e:
            assert e.status in (INVALID, ALIGN, UNSUP)
            continue
        accepted += 1

        def cells(p, rows, cols, pitch):
            return {p + 2 * (r * pitch + c) for r in range(rows) for c in range(cols)} if p else set()

        kn = a["layout"] == "kn"
        x = cells(a["X"], M, K, a["ldx"])
        w = cells(a["W"], K if kn else N, N if kn else K, a["ldw"])
        y, z, r = (cells(a[k], M, N, a[p]) for k, p in (("Y", "ldy"), ("z", "ldz"), ("residual", "ldr")))
        assert not (y & x) and not (y & w) and not (z & (x | w | y | r))
        assert not (y & r) or (a["Y"] == a["residual"] and a["ldy"] == a["ldr"])
        if K:
            assert a["X"] % 16 == 0 and a["W"] % 16 == 0 and a["ldx"] % 8 == 0 and a["ldw"] % 8 == 0
    assert accepted > 100
