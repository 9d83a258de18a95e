"""The clipped policy loss and its gradient against the formulas in float64.

Bounds, from float32 arithmetic: x c - shift carries 2^-23 (|x| + |max|) c of rounding, the sums of
exponentials 2^-21 relative over a tree, so log probabilities are within 2^-20 (2 + |x| + |max|)
absolute and softmax values within 2^-19 (2 + |x| + |max|) relative; a gradient adds half an ulp of
its type, statistics what an error of logp makes of them.
"""
import math

import pytest
import torch

import gg_inputs

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
MANT = {F16: 10, BF16: 7, F32: 23}
FILL = 55.0


def half_ulp(x, dtype):
    ax = torch.clamp_min(x.abs(), 2.0 ** (-14 if dtype == F16 else -126))
    return torch.exp2(torch.floor(torch.log2(ax)) - MANT[dtype] - 1)


def reference(c, logits=None, targets=None):
    """(stats, logp, dlogits) in float64 from the formulas."""
    x = (c["logits"] if logits is None else logits).double() * c["it"]
    t = c["target"].clamp(0, x.shape[1] - 1)
    on = (c["weight"] != 0) & (c["target"] >= 0) & (c["target"] < x.shape[1])
    x = torch.where(on[:, None], x, torch.zeros_like(x))
    logp_all = torch.log_softmax(x, 1)
    logp = logp_all.gather(1, t[:, None])[:, 0]
    A, w = c["adv"].double(), torch.where(on, c["weight"], 0.0).double()
    r = torch.exp(logp - c["old"].double()) if c["old"] is not None else torch.ones_like(logp)
    clip = ((A > 0) & (r > 1 + c["hi"])) | ((A < 0) & (r < 1 - c["lo"]))
    loss = -torch.minimum(r * A, r.clamp(1 - c["lo"], 1 + c["hi"]) * A)
    slope = torch.where(clip, torch.zeros_like(r), -A * r)
    kl = torch.zeros_like(r)
    if c["ref"] is not None and c["kl"]:
        d = c["ref"].double() - logp
        kl = torch.exp(d) - d - 1
        loss = loss + c["kl"] * kl
        slope = slope + c["kl"] * (1 - torch.exp(d))

    def total(q):
        return torch.where(on, w * q, torch.zeros_like(w)).sum()

    stats = torch.stack([total(loss), total(kl), total(clip.double()), total(r)])
    coef = torch.where(on, w * slope, torch.zeros_like(w)) * c["it"] * c["gs"]
    grad = -coef[:, None] * logp_all.exp()
    grad.scatter_add_(1, t[:, None], coef[:, None])
    return stats, torch.where(on, logp, torch.zeros_like(logp)), torch.where(on[:, None], grad, torch.zeros_like(grad))


def make(T, V, dtype, pad=0, shift=0, masked=0.3, old=True, kl=0.05, seed=0, scale=3.0, it=1.0):
    gen = gg_inputs.generator(seed)
    ld = V + pad
    buf = torch.full((T * ld + shift,), FILL, dtype=dtype)
    view = buf[shift:].view(T, ld)[:, :V]
    view.copy_(torch.randn((T, V), generator=gen) * scale)
    dev = buf.cuda()
    c = dict(it=it, lo=0.2, hi=0.28, kl=kl, gs=64.0 if dtype == F16 else 1.0, dtype=dtype, T=T, V=V, ld=ld)
    c["logits"] = dev[shift:].view(T, ld)[:, :V]
    c["target"] = torch.randint(0, V, (T,), generator=gen).cuda()
    lp = torch.log_softmax(c["logits"].double() * it, 1).gather(1, c["target"][:, None])[:, 0]
    noise = torch.randn((3, T), generator=gen).cuda()
    c["old"] = (lp + 0.25 * noise[0]).float() if old else None
    c["ref"] = (lp + 0.4 * noise[1]).float() if kl else None
    c["adv"] = noise[2].contiguous()
    c["weight"] = torch.where(torch.rand((T,), generator=gen) < masked, 0.0, 0.5 + torch.rand((T,), generator=gen)).cuda()
    return c


def call(c, inplace=False, grad=True, gshift=0, gpad=0, stats=True, **kw):
    import gemm_gather_gb300 as gg
    T, V = c["T"], c["V"]
    out = None
    if inplace:
        out = c["logits"]
    elif grad:
        ld = V + gpad
        out = torch.full((T * ld + gshift,), FILL, dtype=c["dtype"], device="cuda")[gshift:].view(T, ld)[:, :V]
    st = torch.full((4,), math.nan, device="cuda") if stats else None
    logp = torch.full((T,), math.nan, device="cuda")
    gg.policy_loss(c["logits"], c["ld"], c["target"], c["old"], c["ref"], c["adv"], c["weight"], T, V,
                   c["dtype"], st, logp, out, out.stride(0) if out is not None else 0,
                   inv_temperature=c["it"], clip_low=c["lo"], clip_high=c["hi"], kl_coef=c["kl"],
                   grad_scale=c["gs"], **kw)
    return st, logp, out


def check(c, got, logits=None):
    stats, logp, grad = got
    want_s, want_l, want_g = reference(c, logits)
    x = (c["logits"] if logits is None else logits).double() * c["it"]
    size = 2 + 2 * x.abs().amax(1)
    e = 2.0 ** -20 * size                      # of a log probability
    assert ((logp.double() - want_l).abs() <= e + 2.0 ** -22 * want_l.abs()).all()
    if stats is not None:
        # every term moves by at most (ratio |A| + kl_coef (1 + exp d) + 1 + exp d + ratio) e
        r = torch.exp(want_l - c["old"].double()) if c["old"] is not None else torch.ones_like(want_l)
        d = torch.exp(c["ref"].double() - want_l) if c["ref"] is not None else torch.zeros_like(want_l)
        w = c["weight"].double()
        per = w * ((r * (c["adv"].double().abs() + 1) + 2 + 2 * d) * (e + 2.0 ** -21 * 4))
        assert ((stats.double() - want_s).abs()[[0, 1, 3]] <= per.sum() + 2.0 ** -22 * w.sum()).all()
        edge = ((r - 1 - c["hi"]).abs().minimum((r - 1 + c["lo"]).abs()) <= 4 * e * r)
        assert (stats.double() - want_s).abs()[2] <= (w * edge).sum() + 2.0 ** -22 * w.sum()
    if grad is not None:
        slack = 2.0 ** -18 * size[:, None] * (want_g.abs() + torch.zeros_like(want_g).scatter_(
            1, c["target"].clamp(0, c["V"] - 1)[:, None], want_g.abs().amax(1, keepdim=True)))
        # dloss/dlogp itself is a difference of terms: its error in units of each term
        A, r = c["adv"].double().abs(), (torch.exp(want_l - c["old"].double()) if c["old"] is not None else 1.0)
        d = torch.exp(c["ref"].double() - want_l) if c["ref"] is not None else 0.0
        coef = c["weight"].double() * (A * r + c["kl"] * (1 + d)) * c["it"] * c["gs"]
        p = torch.softmax(x, 1)
        p.scatter_(1, c["target"].clamp(0, c["V"] - 1)[:, None], 1.0)
        slack = slack + (coef * 4 * (e + 2.0 ** -21))[:, None] * p
        assert ((grad.double() - want_g).abs() <= slack + 1.01 * half_ulp(want_g, c["dtype"])).all()


def far_from_clip(c):
    """Move old_logp where a ratio sits so near a clip edge that rounding decides."""
    if c["old"] is None:
        return c
    _, lp, _ = reference(c)
    r = torch.exp(lp - c["old"].double())
    near = ((r - 1 - c["hi"]).abs() < 1e-3) | ((r - 1 + c["lo"]).abs() < 1e-3)
    c["old"] = torch.where(near, c["old"] + 0.05, c["old"])
    return c


SHAPES = [(1, 1), (3, 2), (1, 7), (5, 63), (7, 129), (2, 1000), (300, 257), (9, 4097), (1, 16384), (2, 32003),
          (40, 20011), (700, 5000), (3, 100003)]


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("T,V", SHAPES)
def test_values(T, V, dtype):
    c = far_from_clip(make(T, V, dtype, pad=(T * 3 + V) % 9, masked=0.3 if T > 4 else 0.0, seed=T + V))
    got = call(c, gpad=3)
    check(c, got)
    full = got[2].as_strided((T, V + 3), (V + 3, 1))
    assert (full[:, V:] == FILL).all()


@pytest.mark.parametrize("T,V,dtype,inplace", [(2, 530001, BF16, False), (3, 600000, F16, True), (2, 270003, F32, False)])
def test_rows_that_no_cluster_holds(T, V, dtype, inplace):
    c = far_from_clip(make(T, V, dtype, pad=V % 2, masked=0.0, seed=8))
    before = c["logits"].clone()
    check(c, call(c, inplace=inplace), before)


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("shift,gshift", [(0, 0), (1, 1), (3, 1), (0, 5)])
def test_alignment_and_in_place(shift, gshift, dtype):
    for V in (1531, 9000):
        c = far_from_clip(make(33, V, dtype, shift=shift, seed=1))
        apart = call(c, gshift=gshift)
        check(c, apart)
        before = c["logits"].clone()
        c2 = dict(c)
        got = call(c2, inplace=True)
        assert all(torch.equal(a, b) for a, b in zip(got, apart))
        check(c, got, before)


@pytest.mark.parametrize("old,kl", [(True, 0.0), (False, 0.05), (False, 0.0)])
@pytest.mark.parametrize("it", [0.5, 1.7])
def test_options(old, kl, it):
    c = far_from_clip(make(50, 777, BF16, old=old, kl=kl, it=it, seed=2))
    got = call(c)
    check(c, got)
    s, lp, g = call(c, grad=False, stats=False)  # the log probabilities alone
    assert s is None and g is None and torch.equal(lp, got[1])


def test_gradient_against_differences():
    """dlogits against central differences of the float64 loss at single logits."""
    c = far_from_clip(make(6, 19, F32, masked=0.2, seed=3))
    _, _, g = call(c)
    x = c["logits"].double()
    for t in range(6):
        for v in range(0, 19, 3):
            d = []
            for s in (1e-5, -1e-5):
                y = x.clone()
                y[t, v] += s
                d.append(float(reference(c, y)[0][0]))
            assert abs((d[0] - d[1]) / 2e-5 - float(g[t, v])) <= 1e-5 * (1 + float(g.abs().max()))


def test_masked_rows_are_not_read():
    import gemm_gather_gb300 as gg
    c = far_from_clip(make(20, 500, BF16, masked=0.0, seed=4))
    off = [0, 7, 19]
    c["weight"][off] = 0
    want = call(c)
    for k in ("old", "ref", "adv"):
        c[k][off] = math.nan
    c["logits"][off] = math.nan
    c["target"][off] = torch.tensor([-100, 10 ** 12, 500], device="cuda")
    got = call(c)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert (got[2][off] == 0).all() and (got[1][off] == 0).all()
    assert gg.device_status() == 0
    c["weight"][:] = 0
    s, lp, g = call(c)
    assert (s == 0).all() and (lp == 0).all() and (g == 0).all()


def test_targets_out_of_range_are_reported():
    c = far_from_clip(make(8, 100, F32, masked=0.0, seed=5))
    c["target"][2], c["target"][5] = -1, 100
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = call(c, status=status)
    assert int(status.item()) == -1
    check(c, got)
    assert (got[2][[2, 5]] == 0).all()


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_infinities_and_nan(dtype):
    c = make(6, 3000, dtype, masked=0.0, seed=6)
    x = c["logits"]
    x[0, 5:2900] = -math.inf                    # a masked vocabulary
    c["target"][0] = 2
    x[1, :] = -math.inf                         # nothing left
    x[2, 17] = math.nan
    x[3, 17] = math.inf
    x[4, :] = torch.finfo(dtype).min            # the type's lowest value everywhere: uniform
    x[5, 1:] = torch.finfo(dtype).min
    c["target"][5] = 0
    c["old"] = c["ref"] = None
    c["kl"] = 0.0
    s, lp, g = call(c)
    for t in (1, 2, 3):
        assert g[t].isnan().all() and lp[t].isnan()
    assert s[0].isnan() and s[3].isnan()        # exp(logp - logp) of a row without a logp
    _, want_l, want_g = reference(c)
    keep = [0, 4, 5]
    assert ((lp.double() - want_l)[keep].abs() <= 2.0 ** -18).all()
    assert (g[0, 5:2900] == 0).all()
    assert ((g.double() - want_g)[keep].abs() <= 2.0 ** -16 * c["adv"].abs().max() * 2 * c["gs"]
            + 1.01 * half_ulp(want_g, dtype)[keep]).all()
    assert abs(float(lp[4]) + math.log(3000)) <= 2.0 ** -18 and lp[5] == 0


def test_no_tokens_and_same_bits():
    import gemm_gather_gb300 as gg
    st = torch.full((4,), 9.0, device="cuda")
    gg.policy_loss(None, 8, None, None, None, None, None, 0, 8, F16, st, None, None, 0)
    assert (st == 0).all()
    c = make(64, 12345, BF16, seed=7)
    a = call(c)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b = call(c)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("T,V", [(300, 4096), (5, 4097), (400, 100003)])
def test_a_wait_that_runs_out_is_reported(T, V):
    """One message of the first token's cluster is never sent: the bounded wait gives up, the status
    word says so, and the same call afterwards is right."""
    import gemm_gather_gb300 as gg
    c = far_from_clip(make(T, V, BF16, masked=0.0, seed=11))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    old = gg.get_wait_limit_ns()
    try:
        gg.set_wait_limit_ns(20_000_000)
        gg.debug_inject_stall(True)
        call(c, status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == -6
    finally:
        gg.debug_inject_stall(False)
        gg.set_wait_limit_ns(old)
    status.zero_()
    got = call(c, status=status)
    assert int(status.item()) == 0
    check(c, got)
