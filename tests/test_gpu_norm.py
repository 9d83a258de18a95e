"""The root-mean-square norm and its gradients against float64.

h is the sum rounded once, so equal bit by bit.  rstd: the squares are summed in float32, a thread's at
most 32 (rows that are read once) or N / 512 + 1 one after the other and then some 11 in a tree, all of
one sign, so its relative error is half of (N / 512 + 45) 2^-24, plus the division, root and addition:
(N / 1024 + 26) 2^-24.  y: that, two products, and half an ulp.  The codes are those of the y that was
given, bit by bit.  dh and dweight: each sum's own bound of the same kind times the sum of magnitudes
(a column's sum has M terms in a chain at most), and half an ulp of the output.
"""
import pytest
import torch

import gemm_gather_gb300 as gg
from tests import block_oracle as o
from tests.block_oracle import BF16, F16, F32

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn
SIZES = [(1, 8192), (1, 1), (1, 31), (3, 64), (5, 1000), (7, 1523), (200, 128), (333, 136), (777, 1523), (40, 4096),
         (311, 8192), (153, 16384), (9, 32768), (4, 40000), (700, 257), (2000, 8)]


def bits(x):
    return x.contiguous().view(torch.int16)


def make(M, N, dtype, seed=0, wdtype=None, residual=True, pad=0, shift=0):
    g = torch.Generator().manual_seed(seed + 7 * M + N)
    x, r = torch.randn((M, N), generator=g) * 1.5, torch.randn((M, N), generator=g) * 0.5
    w = (1 + 0.2 * torch.randn((N,), generator=g)).to(wdtype or dtype).cuda()
    return o.put(x, dtype, pad, shift), o.put(r, dtype, pad, shift) if residual else None, w


def codes_room(M, N, pad=0, shift=0):
    ld = (N + 15) // 16 * 16 + pad
    buf = torch.full((M * ld + shift,), 3, dtype=torch.uint8, device="cuda")
    return buf[shift:].as_strided((M, N), (ld, 1), shift).view(E4M3)


def norm(x, r, w, eps=1e-6, h=None, y=None, codes=None, scales=None, rstd=None, **kw):
    ld = lambda t: t.stride(0) if t is not None else 0   # noqa: E731
    M, N = x.shape
    gg.rms_norm(x, ld(x), r, ld(r), w, eps, h, ld(h), y, ld(y), codes, ld(codes), scales, ld(scales), rstd, M, N,
                x.dtype, **kw)


def check_norm(x, r, w, eps, h, y, codes, scales, rstd, x_before=None, r_before=None):
    x, r = x if x_before is None else x_before, r if r_before is None else r_before
    M, N = x.shape
    dt = x.dtype
    total = (x.float() + r.float()).to(dt) if r is not None else x
    if h is not None:
        assert torch.equal(bits(h), bits(total))
    t = total.double()
    want = 1 / torch.sqrt(t.square().mean(1) + eps)
    if rstd is not None:
        assert ((rstd.double() - want).abs() <= want * (N / 1024 + 26) * 2.0 ** -24).all()
    wy = t * want[:, None] * w.double()
    if y is not None:
        assert ((y.double() - wy).abs() <= wy.abs() * (N / 1024 + 30) * 2.0 ** -24 + o.half_ulp(wy, dt) * 1.001).all()
        if codes is not None:
            c, s = o.pack(y)
            assert torch.equal(scales.double(), s)
            assert torch.equal(codes.double(), c)


@pytest.mark.parametrize("M,N", SIZES)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_forward(M, N, dtype):
    x, r, w = make(M, N, dtype, wdtype=F32 if N % 2 else dtype, residual=M % 3 != 1)
    h, y = o.room(M, N, dtype), o.room(M, N, dtype, pad=8)
    codes, scales = codes_room(M, N), o.room(M, -(-N // 128), F32, pad=1)
    rstd = torch.empty((M,), device="cuda")
    norm(x, r, w, h=h, y=y, codes=codes, scales=scales, rstd=rstd)
    check_norm(x, r, w, 1e-6, h, y, codes, scales, rstd)
    assert o.untouched(h) and o.untouched(y) and o.untouched(scales)
    assert bool((o.rest(codes.view(torch.uint8)) == 3).all())


@pytest.mark.parametrize("M,N", [(1, 100), (50, 1523), (300, 4096), (3, 40000)])
@pytest.mark.parametrize("pad,shift", [(1, 0), (0, 1), (3, 5)])
def test_forward_any_alignment(M, N, pad, shift):
    x, r, w = make(M, N, BF16, pad=pad, shift=shift)
    h, y = o.room(M, N, BF16, pad, shift), o.room(M, N, BF16, pad, shift)
    codes, scales, rstd = codes_room(M, N, pad, shift), o.room(M, -(-N // 128), F32, pad, shift), torch.empty((M,), device="cuda")
    norm(x, r, w, h=h, y=y, codes=codes, scales=scales, rstd=rstd)
    check_norm(x, r, w, 1e-6, h, y, codes, scales, rstd)
    assert o.untouched(h) and o.untouched(y)
    # weights that start anywhere
    buf = torch.zeros((N + 1,), dtype=BF16, device="cuda")
    buf[1:] = w
    y2 = o.room(M, N, BF16)
    x2 = o.put(x, BF16)
    norm(x2, o.put(r, BF16), buf[1:], y=y2)
    check_norm(x, r, w, 1e-6, None, y2, None, None, None)


@pytest.mark.parametrize("pad", [0, 1])
@pytest.mark.parametrize("N", [200, 2048, 40000])
def test_forward_in_place(N, pad):
    M = 37
    for hx, yx in ((True, False), (False, True), (True, True), (False, None)):
        x, r, w = make(M, N, F16, pad=pad)
        x0, r0 = x.clone(), r.clone()
        h = x if hx else r
        y = None if yx is None else (r if yx else x)
        if h is y:
            h = None
        y = o.room(M, N, F16, pad) if y is None else y
        codes, scales = codes_room(M, N), torch.empty((M, -(-N // 128)), device="cuda")
        norm(x, r, w, h=h, y=y, codes=codes, scales=scales)
        check_norm(x, r, w, 1e-6, h, y, codes, scales, None, x0, r0)


def test_forward_codes_alone_and_y_alone():
    x, r, w = make(64, 1000, BF16)
    y, c1, s1 = o.room(64, 1000, BF16), codes_room(64, 1000), torch.empty((64, 8), device="cuda")
    c2, s2 = codes_room(64, 1000), torch.empty((64, 8), device="cuda")
    norm(x, r, w, y=y, codes=c1, scales=s1)
    norm(x, r, w, codes=c2, scales=s2)
    assert torch.equal(c1.view(torch.uint8), c2.view(torch.uint8)) and torch.equal(s1, s2)
    c3, s3 = codes_room(64, 1000), torch.empty((64, 8), device="cuda")
    gg.pack8(y, y.stride(0), c3, c3.stride(0), s3, 8, 64, 1000, BF16)
    assert torch.equal(c1.view(torch.uint8), c3.view(torch.uint8)) and torch.equal(s1, s3)


@pytest.mark.parametrize("pad", [0, 1])
def test_forward_rows_that_are_not_ordinary(pad):
    """Zeros (with and without eps), NaN and infinities, sizes whose squares are subnormal or overflow."""
    N = 300
    x, _, w = make(8, N, BF16, residual=False, pad=pad)
    x[0] = 0
    x[1, 17] = float("nan")
    x[2, 5] = float("inf")
    x[3, 250] = -float("inf")
    x[4] *= 1e-30
    x[5] *= 1e25
    for eps in (1e-6, 0.0):
        y, rstd = o.room(8, N, BF16, pad), torch.empty((8,), device="cuda")
        codes, scales = codes_room(8, N), torch.empty((8, 3), device="cuda")
        norm(x, None, w, eps=eps, y=y, codes=codes, scales=scales, rstd=rstd)
        if eps:
            assert (y[0] == 0).all() and (codes[0].double() == 0).all() and abs(float(rstd[0]) - 1000) < 1e-2
        else:
            assert y[0].isnan().all() and codes[0].float().isnan().all()
        assert y[1].isnan().all() and rstd[1].isnan()
        for k in (2, 3):   # inf / inf where it is, 0 elsewhere
            assert y[k].isnan().sum() == 1 and float(rstd[k]) == 0 and (y[k].nan_to_num() == 0).all()
            assert codes[k].float().isnan().sum() == 1
        if eps:
            t = x[4].double() * w.double() * 1000
            assert ((y[4].double() - t).abs() <= t.abs() * 2.0 ** -7.9 + 1e-40).all()
        assert float(rstd[5]) == 0
        check_norm(x[6:], None, w, eps, None, y[6:], codes[6:], scales[6:], rstd[6:])


def test_nothing_to_do():
    w = torch.ones((64,), dtype=BF16, device="cuda")
    y = torch.full((4, 64), 5.0, dtype=BF16, device="cuda")
    gg.rms_norm(y, 64, None, 0, w, 1e-6, None, 0, y, 64, None, 0, None, 0, None, 0, 64, BF16)
    gg.rms_norm(y, 64, None, 0, w, 1e-6, None, 0, y, 64, None, 0, None, 0, None, 4, 0, BF16)
    assert (y == 5).all()
    dw = torch.full((64,), 3.0, device="cuda")
    rstd = torch.ones((4,), device="cuda")
    for acc, want in ((True, 3.0), (False, 0.0)):
        gg.rms_norm_backward(None, 64, None, 64, None, None, None, 0, None, 0, dw, F32, acc, None, 0, 64, BF16)
        assert (dw == want).all()
    gg.rms_norm_backward(y, 64, y, 64, rstd, w, None, 0, None, 0, None, F32, False, None, 4, 64, BF16)


# ---- gradients ------------------------------------------------------------------------------------
def backward(dy, h, rstd, w, dh_in, dh, dw, accumulate=False, workspace=None, **kw):
    ld = lambda t: t.stride(0) if t is not None else 0   # noqa: E731
    M, N = dy.shape
    need = gg.rms_norm_backward_workspace(M, N)
    room = torch.full((need + 64,), 0xEE, dtype=torch.uint8, device="cuda") if workspace is None else workspace
    gg.rms_norm_backward(dy, ld(dy), h, ld(h), rstd, w, dh_in, ld(dh_in), dh, ld(dh), dw,
                         dw.dtype if dw is not None else F32, accumulate, room, M, N, dy.dtype, workspace_bytes=need, **kw)
    if workspace is None:
        assert (room[need:] == 0xEE).all()


def gradients64(dy, h, rstd, w, dh_in):
    dy, h, w, r = dy.double(), h.double(), w.double(), rstd.double()[:, None]
    u, g = h * r, dy * w
    dh = r * (g - u * (g * u).mean(1, keepdim=True))
    size = r.abs() * (g.abs() + u.abs() * (g * u).abs().mean(1, keepdim=True))
    if dh_in is not None:
        dh, size = dh + dh_in.double(), size + dh_in.double().abs()
    return dh, size, (dy * u).sum(0), (dy * u).abs().sum(0)


def check_gradients(dy, h, rstd, w, dh_in, dh, dw, before=None):
    M, N = dy.shape
    want, size, ww, wsize = gradients64(dy, h, rstd, w, dh_in)
    if dh is not None:
        assert ((dh.double() - want).abs() <= size * (N / 512 + 52) * 2.0 ** -24 + o.half_ulp(want, dy.dtype) * 1.01).all()
    if dw is not None:
        if before is not None:
            ww, wsize = ww + before.double(), wsize + before.double().abs()
        assert ((dw.double() - ww).abs() <= wsize * (M + 16) * 2.0 ** -24 + o.half_ulp(ww, dw.dtype) * 1.01).all()


def make_backward(M, N, dtype, wdtype, through, pad=0, shift=0):
    h, dh_in, w = make(M, N, dtype, 1, wdtype, True, pad, shift)
    g = torch.Generator().manual_seed(M + N)
    dy = o.put(torch.randn((M, N), generator=g) * 0.1, dtype, pad, shift)
    rstd = torch.rsqrt(h.double().square().mean(1) + 1e-6).float()
    return dy, h, rstd, w, dh_in if through else None


@pytest.mark.parametrize("M,N", SIZES + [(3000, 96), (1000, 2048)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_backward(M, N, dtype):
    through, grad, acc = N % 3 != 0, F32 if M % 2 else dtype, M % 3 == 0
    dy, h, rstd, w, dh_in = make_backward(M, N, dtype, F32 if N % 2 else dtype, through)
    dh = o.room(M, N, dtype, pad=8)
    dw = torch.randn((N,), device="cuda").to(grad)
    before = dw.clone() if acc else None
    backward(dy, h, rstd, w, dh_in, dh, dw, acc)
    check_gradients(dy, h, rstd, w, dh_in, dh, dw, before)
    assert o.untouched(dh)
    # either alone, the same bits
    dh2, dw2 = o.room(M, N, dtype), before.clone() if acc else torch.empty_like(dw)
    backward(dy, h, rstd, w, dh_in, dh2, None)
    backward(dy, h, rstd, w, None, None, dw2, acc)
    assert torch.equal(bits(dh), bits(dh2)) and torch.equal(dw, dw2)


@pytest.mark.parametrize("M,N", [(1, 100), (50, 1523), (300, 2048), (3, 40000)])
@pytest.mark.parametrize("pad,shift", [(1, 0), (0, 1)])
def test_backward_any_alignment(M, N, pad, shift):
    dy, h, rstd, w, dh_in = make_backward(M, N, F16, F16, True, pad, shift)
    dh, dw = o.room(M, N, F16, pad, shift), torch.empty((N,), device="cuda")
    backward(dy, h, rstd, w, dh_in, dh, dw)
    check_gradients(dy, h, rstd, w, dh_in, dh, dw)
    assert o.untouched(dh)


@pytest.mark.parametrize("pad", [0, 1])
@pytest.mark.parametrize("N", [200, 4096, 33000])
@pytest.mark.parametrize("over", ["dy", "h", "dh_in"])
def test_backward_in_place(N, pad, over):
    dy, h, rstd, w, dh_in = make_backward(65, N, BF16, BF16, True, pad)
    b = {"dy": dy.clone(), "h": h.clone(), "dh_in": dh_in.clone()}
    dh, dw = {"dy": dy, "h": h, "dh_in": dh_in}[over], torch.empty((N,), device="cuda")
    backward(dy, h, rstd, w, dh_in, dh, dw)
    check_gradients(b["dy"], b["h"], rstd, w, b["dh_in"], dh, dw)


def test_backward_against_differences():
    """The kernel's gradients against central differences of the forward formula in float64."""
    M, N, eps = 4, 24, 1e-3
    dy, h, _, w, _ = make_backward(M, N, BF16, F32, False)
    rstd = torch.rsqrt(h.double().square().mean(1) + eps).float()
    dh, dw = o.room(M, N, BF16), torch.empty((N,), device="cuda")
    backward(dy, h, rstd, w, None, dh, dw)

    def f(h, w):
        return (h / torch.sqrt(h.square().mean(1, keepdim=True) + eps) * w * dy.double()).sum()
    h64, w64, d = h.double(), w.double(), 1e-5
    for m in range(M):
        for n in range(0, N, 5):
            e = torch.zeros_like(h64)
            e[m, n] = d
            slope = float((f(h64 + e, w64) - f(h64 - e, w64)) / (2 * d))
            # half an ulp of the output, and float32 sums of 24 terms
            assert abs(float(dh[m, n]) - slope) <= abs(slope) * 2.0 ** -7.9 + 1e-6
    for n in range(N):
        e = torch.zeros_like(w64)
        e[n] = d
        slope = float((f(h64, w64 + e) - f(h64, w64 - e)) / (2 * d))
        assert abs(float(dw[n]) - slope) <= 1e-5 * abs(slope) + 1e-6


def test_on_another_stream_and_in_a_graph():
    dy, h, rstd, w, dh_in = make_backward(500, 2048, BF16, BF16, True)
    x, r, _ = make(500, 2048, BF16)
    y, hh, dh = (o.room(500, 2048, BF16) for _ in range(3))
    dw, rs = torch.empty((2048,), device="cuda"), torch.empty((500,), device="cuda")
    room = torch.empty((gg.rms_norm_backward_workspace(500, 2048),), dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        norm(x, r, w, h=hh, y=y, rstd=rs)
        backward(dy, hh, rs, w, dh_in, dh, dw, workspace=room)
    s.synchronize()
    want = [t.clone() for t in (y, hh, dh, dw, rs)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        norm(x, r, w, h=hh, y=y, rstd=rs)
        backward(dy, hh, rs, w, dh_in, dh, dw, workspace=room)
    for t in (y, hh, dh, dw, rs):
        t.zero_()
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    for t, u in zip((y, hh, dh, dw, rs), want):
        assert torch.equal(t, u)
