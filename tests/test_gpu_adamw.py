"""AdamW against the formulas in float64, and its 8-bit states against their definition.

32-bit states: a handful of float32 operations, each within 2^-24 relative, so m and v within 2^-21
of the sizes of their terms; the parameter within 2^-23 of itself and 2^-20 of the update.
8-bit states: a code is one of the two e4m3 neighbours of the exact value (of a float32's nearness to
it), the scale its block's power of two, and rounding is right on average.
"""
import math

import pytest
import torch

import gg_inputs

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
MANT = {F16: 10, BF16: 7, F32: 23}
HYPER = dict(lr=1e-2, beta1=0.9, beta2=0.99, eps=1e-6, weight_decay=0.1)
BLOCK = 256


def half_ulp(x, dtype):
    ax = torch.clamp_min(x.abs(), 2.0 ** (-14 if dtype == F16 else -126))
    return torch.exp2(torch.floor(torch.log2(ax)) - MANT[dtype] - 1)


def place(x, shift):
    """x on the GPU, `shift` elements behind a 16-byte boundary, with a guard element after it."""
    buf = torch.zeros((x.numel() + shift + 1,), dtype=x.dtype, device="cuda")
    buf[shift:shift + x.numel()] = x
    buf[shift + x.numel()] = 3
    return buf[shift:shift + x.numel()], buf


def scale_of(top):
    """2^k with top / 2^k in (224, 448], k >= -118."""
    if top == 0:
        return 2.0 ** -118
    f, e = math.frexp(top)                       # top = f 2^e, f in [0.5, 1)
    return 2.0 ** max(e - 9 + (f > 0.875), -118)


def make(n, param=F32, grad=F32, bits=32, copy=None, shift=0, gen=None, m_size=3e-3):
    gen = gen or gg_inputs.generator(n)

    def r(scale):
        return torch.randn((n,), generator=gen) * scale

    t, guards = {}, {}
    vals = {"param": r(0.5).to(param), "grad": r(0.1).to(grad), "m": r(m_size), "v": r(0.1).square() + 1e-6}
    if bits == 8:
        for k in ("m", "v"):
            x = vals[k] if k == "m" else vals[k].sqrt()
            sc = torch.tensor([scale_of(float(b.abs().max())) for b in x.split(BLOCK)])
            vals[k] = (x / sc.repeat_interleave(BLOCK)[:n]).to(torch.float8_e4m3fn).view(torch.uint8)
            t[k + "_scale"] = sc.cuda()
    if copy is not None:
        vals["copy"] = torch.zeros((n,), dtype=copy)
    for k, x in vals.items():
        t[k], guards[k] = place(x, shift)
    t["guards"] = guards
    return t


def values(t, k):
    """What a state stands for, in float64."""
    x = t[k]
    if x.dtype == torch.uint8:
        x = x.view(torch.float8_e4m3fn).double() * t[k + "_scale"].double().repeat_interleave(BLOCK)[:x.numel()]
        return x if k == "m" else x.square()
    return x.double()


def expected(t, step, gs=1.0, h=HYPER):
    g = t["grad"].double() * gs
    m = h["beta1"] * values(t, "m") + (1 - h["beta1"]) * g
    v = h["beta2"] * values(t, "v") + (1 - h["beta2"]) * g * g
    mh, vh = m / (1 - h["beta1"] ** step), v / (1 - h["beta2"] ** step)
    upd = h["lr"] * mh / (vh.sqrt() + h["eps"])
    p = t["param"].double()
    return p * (1 - h["lr"] * h["weight_decay"]) - upd, m, v, upd


def run(ts, step, bits, gs=None, seed=7, h=HYPER):
    import gemm_gather_gb300 as gg
    table = gg.adamw_tensors(ts, state_bits=bits)
    scale = torch.full((1,), gs, device="cuda") if gs is not None else None
    gg.adamw(table, step, grad_scale=scale, seed=seed, **h)
    torch.cuda.synchronize()


def check_params(t, p, upd, before):
    bound = 2.0 ** -22 * (p.abs() + before.double().abs()) + 2.0 ** -19 * upd.abs()
    dt = t["param"].dtype
    assert ((t["param"].double() - p).abs() <= bound + (1.01 * half_ulp(p, dt) if dt != F32 else 0)).all()
    if t.get("copy") is not None:
        want = t["param"].to(t["copy"].dtype)
        assert torch.equal(t["copy"], want)


def check_guards(t):
    for k, g in t["guards"].items():
        assert float(g[-1]) == 3


SIZES = [1, 3, 255, 256, 257, 2048, 2049, 70000]


@pytest.mark.parametrize("param,grad,copy", [(F32, F32, None), (F32, BF16, BF16), (F32, F16, F16), (BF16, BF16, None),
                                             (F16, F32, None), (BF16, F16, None), (F16, BF16, None)])
@pytest.mark.parametrize("shift", [0, 1])
def test_states_of_32_bits(param, grad, copy, shift):
    ts = [make(n, param, grad, 32, copy, shift) for n in SIZES]
    old = [(expected(t, 3, 0.5), t["param"].clone()) for t in ts]
    run(ts, 3, 32, gs=0.5)
    for t, ((p, m, v, upd), before) in zip(ts, old):
        assert ((t["m"].double() - m).abs() <= 2.0 ** -21 * (m.abs() + 0.1 * t["grad"].double().abs())).all()
        assert ((t["v"].double() - v).abs() <= 2.0 ** -21 * v).all()
        check_params(t, p, upd, before)
        check_guards(t)


def neighbours_ok(codes, scale, exact):
    """codes * scale against exact values: off by less than one e4m3 step (of the larger
    neighbour), up to a float32's rounding; a value that is a code stays that code."""
    got = codes.view(torch.float8_e4m3fn).double()
    y = exact / scale.double().repeat_interleave(BLOCK)[:exact.numel()]
    assert (y.abs() <= 448 * (1 + 2.0 ** -22)).all()
    step = torch.exp2(torch.clamp_min(torch.floor(torch.log2(y.abs().clamp_min(1e-30))), -6.0) - 3)
    return ((got - y).abs() <= step * (1 + 2.0 ** -16)).all()


@pytest.mark.parametrize("param,grad,copy", [(F32, BF16, BF16), (BF16, BF16, None), (F32, F32, None), (F16, F16, None)])
@pytest.mark.parametrize("shift", [0, 1])
def test_states_of_8_bits(param, grad, copy, shift):
    ts = [make(n, param, grad, 8, copy, shift) for n in SIZES]
    old = [(expected(t, 3), t["param"].clone()) for t in ts]
    run(ts, 3, 8)
    for t, ((p, m, v, upd), before) in zip(ts, old):
        check_params(t, p, upd, before)
        check_guards(t)
        for k, x in (("m", m), ("v", v.sqrt())):
            assert neighbours_ok(t[k], t[k + "_scale"], x)
            for b, s in zip(x.split(BLOCK), t[k + "_scale"].tolist()):
                top = float(b.abs().max())
                # the scale of a float32 near the exact largest value
                assert s in (scale_of(top), scale_of(top * (1 - 2.0 ** -21)), scale_of(top * (1 + 2.0 ** -21)))


def test_rounding_is_right_on_average():
    """n equal values between two codes: the mean of n independent roundings is within 5 standard
    deviations of a mean of n (step / 2 / sqrt(n) at most), for m and for sqrt(v), at values in
    the normal and the subnormal range of the codes."""
    n = 1 << 16
    h = dict(lr=0.0, beta1=0.0, beta2=0.0, eps=1e-8, weight_decay=0.0)
    for y in (300.0, 17.3, 1.03, 0.0171, 0.0042, 0.0007):
        t = make(n, bits=8)
        t["grad"].fill_(y)
        t["grad"][::BLOCK] = 448.0               # the scale of every block is then 1
        run([t], 1, 8, h=h)
        assert (t["m_scale"] == 1).all() and (t["v_scale"] == 1).all()
        step = 2.0 ** (max(math.floor(math.log2(y)), -6) - 3)
        for k in ("m", "v"):
            got = t[k].view(torch.float8_e4m3fn).double()
            rest = torch.ones(n, dtype=torch.bool, device="cuda")
            rest[::BLOCK] = False
            assert abs(float(got[rest].mean()) - y) <= 5 * step / 2 / math.sqrt(n) + step * 2.0 ** -15


def test_second_moment_follows_small_steps():
    """beta2 = 0.999 and gradients of one size: sqrt(v) comes within 10% of it in 5000 steps.
    Rounded to nearest, it would stop at an eighth of it."""
    n = 4096
    t = make(n, bits=8)
    t["m"].zero_()
    t["v"].zero_()
    t["grad"].fill_(0.5)
    h = dict(lr=0.0, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0)
    import gemm_gather_gb300 as gg
    table = gg.adamw_tensors([t], state_bits=8)
    for k in range(1, 5001):
        gg.adamw(table, k, seed=3, **h)
    assert abs(float(values(t, "v").mean().sqrt()) - 0.5) <= 0.05
    assert abs(float(values(t, "m").mean()) - 0.5) <= 0.01


def test_seed_step_and_position_change_the_rounding():
    a, b, c, d = (make(5000, bits=8, gen=gg_inputs.generator(1)) for _ in range(4))
    run([a], 5, 8, seed=1 << 40)
    run([b], 5, 8, seed=1 << 40)
    run([c], 5, 8, seed=1 << 41)
    first = make(10, bits=8)
    run([first, d], 5, 8, seed=1 << 40)
    assert torch.equal(a["m"], b["m"]) and torch.equal(a["v"], b["v"]) and torch.equal(a["param"], b["param"])
    for other in (c, d):
        assert not torch.equal(a["m"], other["m"]) and not torch.equal(a["v"], other["v"])
        assert torch.equal(a["param"], other["param"])


def test_values_that_are_not_finite():
    t = make(600, bits=8)
    t["grad"][3], t["grad"][300], t["grad"][301] = math.nan, math.inf, 1e30
    clean = make(600, bits=8)
    clean["grad"][301] = 1e30
    clean["grad"][3] = clean["grad"][300] = 0.0
    run([t], 2, 8)
    run([clean], 2, 8)
    m, v = values(t, "m"), values(t, "v")
    assert m[3].isnan() and v[3].isnan() and m[300].isnan() and v[300].isnan()
    keep = torch.ones(600, dtype=torch.bool, device="cuda")
    keep[[3, 300]] = False
    assert torch.equal(t["m"][keep], clean["m"][keep]) and torch.equal(t["m_scale"], clean["m_scale"])
    assert t["param"][3].isnan() and torch.equal(t["param"][keep], clean["param"][keep])


def test_many_tensors_of_mixed_types():
    """More tensors than a launch takes, of several types in one list, empty ones among them."""
    import ctypes
    import gemm_gather_gb300 as gg
    kinds = [(F32, F32, 32), (BF16, BF16, 32), (F32, BF16, 8), (F16, F32, 8)]
    ts = [make(1 + 37 * i % 900, *kinds[i % 4][:2], kinds[i % 4][2], gen=gg_inputs.generator(i)) for i in range(1100)]
    old = [(expected(t, 9), t["param"].clone()) for t in ts]
    tables = [gg.adamw_tensors([t], state_bits=kinds[i % 4][2]) for i, t in enumerate(ts)]
    array = (gg.AdamwTensor * 1101)()
    for i, t in enumerate(tables):
        array[i if i < 500 else i + 1] = t.array[0]
    array[500].state_bits = 32                     # an empty tensor, all pointers NULL
    assert ctypes.sizeof(gg.AdamwTensor) == 80
    gg.adamw(gg.AdamwTensors(array, ts), 9, seed=1, **HYPER)
    torch.cuda.synchronize()
    for i, (t, ((p, m, v, upd), before)) in enumerate(zip(ts, old)):
        check_params(t, p, upd, before)
        if kinds[i % 4][2] == 32:
            assert ((t["v"].double() - v).abs() <= 2.0 ** -21 * v).all()
        else:
            assert neighbours_ok(t["m"], t["m_scale"], m)


def test_zero_gradients_and_graph():
    t = make(1000, F32, F32, 32)
    t["grad"].zero_()
    t["m"].zero_()
    t["v"].zero_()
    before = t["param"].clone()
    run([t], 1, 32)
    assert ((t["param"] - before * (1 - 1e-3)).abs() <= 2.0 ** -22 * before.abs()).all()
    import gemm_gather_gb300 as gg
    a, b = make(5000, F32, BF16, 8, BF16), make(5000, F32, BF16, 8, BF16)
    ta, tb = gg.adamw_tensors([a], 8), gg.adamw_tensors([b], 8)
    gg.adamw(ta, 4, seed=2, **HYPER)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gg.adamw(tb, 4, seed=2, **HYPER)
    graph.replay()
    torch.cuda.synchronize()
    for k in ("param", "m", "v", "m_scale", "v_scale", "copy"):
        assert torch.equal(a[k], b[k])


@pytest.mark.parametrize("param,grad,copy", [(F32, BF16, BF16), (BF16, BF16, None), (F32, F32, None)])
def test_8_bit_states_do_not_depend_on_where_the_tensors_lie(param, grad, copy):
    """At a 16-byte boundary, 8 and 4 elements behind one (tensors of a flat buffer) and 1 element:
    the same codes and scales, whichever way the blocks are loaded."""
    first = None
    for shift in (0, 8, 4, 1):
        t = make(70000, param, grad, 8, copy, shift)
        (p, m, v, upd), before = expected(t, 3), t["param"].clone()
        run([t], 3, 8)
        check_params(t, p, upd, before)
        check_guards(t)
        assert neighbours_ok(t["m"], t["m_scale"], m) and neighbours_ok(t["v"], t["v_scale"], v.sqrt())
        got = [t[k].clone() for k in ("m", "v", "m_scale", "v_scale")]
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(first, got))
