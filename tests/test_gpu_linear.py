"""The linear layer and its gradients against plain float64 products.

* Integer-valued operands: every product and partial sum is an exact integer
  in float32, so results must be equal bit for bit, on both kernels, in both
  weight layouts, at ragged sizes, with padding columns untouched.
* Random operands: each value within the float32 summation bound of the
  contraction (K * 2^-23 * sum |x_k w_k|, which also covers an accumulator that
  truncates), scaled by the activation's largest slope, plus 2^-20 of the value
  for the activation's own arithmetic, plus half an ulp of the output type.
* Gradients also against central differences of the forward formula.
"""
import math

import pytest
import torch

import gg_inputs

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
MANT = {F16: 10, BF16: 7, F32: 23}
SLOPE = 1.13          # largest |act'| of the five (gelu: 1.129)
FILL = 77.0           # what padding columns hold before and after


def act64(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return z * 0.5 * (1 + torch.erf(z / math.sqrt(2)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if act == "silu":
        return z * torch.sigmoid(z)
    return z


def slope64(z, act):
    """Central differences of the activation in float64 (relu: its formula)."""
    if act == "relu":
        return (z > 0).double()
    if act == "none":
        return torch.ones_like(z)
    h = 1e-5
    return (act64(z + h, act) - act64(z - h, act)) / (2 * h)


def half_ulp(x, dtype):
    ax = torch.clamp_min(x.abs(), 2.0 ** (-14 if dtype == F16 else -126))
    return torch.exp2(torch.floor(torch.log2(ax)) - MANT[dtype] - 1)


def mat(rows, cols, dtype, gen, ints=False, pad=0, scale=1.0):
    """rows x cols on the GPU with a pitch of whole 16-byte units (+ pad elements)."""
    ld = (cols + 7) // 8 * 8 + pad
    buf = torch.full((rows, ld), FILL, dtype=dtype)
    x = (gg_inputs.integers((rows, cols), -2, 2, F32, gen) if ints
         else torch.randn((rows, cols), generator=gen) * scale)
    buf[:, :cols] = x.to(dtype)
    return buf.cuda()[:, :cols]


def out_mat(rows, cols, dtype, pad=0):
    return torch.full((rows, cols + pad), FILL, dtype=dtype, device="cuda")[:, :cols]


def padding(view):
    """The columns of a view's rows beyond its own."""
    rows, ld = view.shape[0], view.stride(0)
    full = view.as_strided((rows, ld), (ld, 1))
    return full[:, view.shape[1]:]


def weight64(w, layout):
    return w.double() if layout == "kn" else w.double().t()


def call_linear(x, w, layout, bias, act, r, y, z, path="auto", **kw):
    import gemm_gather_gb300 as gg
    M, K = x.shape
    N = w.shape[1] if layout == "kn" else w.shape[0]
    gg.linear(x, x.stride(0), w, w.stride(0), layout, bias, act, r,
              r.stride(0) if r is not None else 0, y, y.stride(0), z,
              z.stride(0) if z is not None else 0, M, N, K, x.dtype, path=path, **kw)


def status_ok():
    import gemm_gather_gb300 as gg
    assert gg.device_status() == 0


SHAPES = [  # (M, N, K)
    (1, 64, 64), (1, 129, 1000), (2, 1, 1), (3, 257, 63), (16, 128, 65), (17, 300, 520), (33, 96, 2048),
    (64, 513, 129), (100, 1000, 72), (128, 128, 64), (129, 255, 200), (255, 256, 128), (257, 511, 577),
    (300, 1000, 1024), (224, 2560, 64), (1020, 3500, 72), (960, 3300, 136),
]


@pytest.mark.parametrize("path", ["split", "pair"])
@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_integers_are_exact(M, N, K, layout, path):
    gen = gg_inputs.generator(M * 7 + N + K)
    dtype = F16 if (M + N) % 2 else BF16
    x = mat(M, K, dtype, gen, ints=True, pad=8)
    w = mat(*((K, N) if layout == "kn" else (N, K)), dtype, gen, ints=True)
    bias = gg_inputs.integers((N,), -2, 2, dtype, gen).cuda()
    r = out_mat(M, N, dtype, 3)
    r.copy_(gg_inputs.integers((M, N), -2, 2, dtype, gen))
    y, z = out_mat(M, N, dtype, 5), out_mat(M, N, dtype, 1)
    call_linear(x, w, layout, bias, "relu", r, y, z, path)
    zr = x.double() @ weight64(w, layout) + bias.double()
    assert torch.equal(z, zr.to(dtype))
    assert torch.equal(y, (zr.clamp_min(0) + r.double()).to(dtype))
    assert (padding(y) == FILL).all() and (padding(z) == FILL).all()
    status_ok()


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("M,N,K,layout,path", [
    (1, 1000, 4096, "nk", "auto"), (27, 515, 777, "kn", "auto"), (70, 260, 1500, "kn", "split"),
    (200, 300, 900, "nk", "pair"), (513, 770, 1030, "kn", "pair")])
def test_random_values(M, N, K, layout, path, dtype, act):
    gen = gg_inputs.generator(11)
    x = mat(M, K, dtype, gen)
    w = mat(*((K, N) if layout == "kn" else (N, K)), dtype, gen, scale=K ** -0.5)
    bias = torch.randn((N,), generator=gen).cuda()  # a float32 bias
    r = mat(M, N, dtype, gen)
    y, z = out_mat(M, N, dtype), out_mat(M, N, dtype)
    call_linear(x, w, layout, bias, act, r, y, z, path)
    z64 = x.double() @ weight64(w, layout) + bias.double()
    err = (K + 4) * 2.0 ** -23 * (x.double().abs() @ weight64(w, layout).abs() + bias.double().abs())
    assert ((z.double() - z64).abs() <= err + half_ulp(z64, dtype) * 1.01).all()
    y64 = act64(z64, act) + r.double()
    bound = SLOPE * err + 2.0 ** -20 * (z64.abs() + r.double().abs()) + half_ulp(y64, dtype) * 1.01
    assert ((y.double() - y64).abs() <= bound).all()
    status_ok()


@pytest.mark.parametrize("path", ["split", "pair"])
def test_optional_arguments_and_in_place_residual(path):
    gen = gg_inputs.generator(5)
    M, N, K, dtype = 150, 203, 130, BF16
    x, w = mat(M, K, dtype, gen, ints=True), mat(N, K, dtype, gen, ints=True)
    p = x.double() @ w.double().t()
    y = out_mat(M, N, dtype)
    call_linear(x, w, "nk", None, "none", None, y, None, path)
    assert torch.equal(y, p.to(dtype))
    y.copy_(gg_inputs.integers((M, N), -2, 2, dtype, gen))
    want = (p + y.double()).to(dtype)
    call_linear(x, w, "nk", None, "none", y, y, None, path)  # the residual is Y itself
    assert torch.equal(y, want)


@pytest.mark.parametrize("path", ["split", "pair"])
@pytest.mark.parametrize("layout", ["kn", "nk"])
def test_empty_sizes(layout, path):
    import gemm_gather_gb300 as gg
    dtype = F16
    bias = torch.arange(-20, 20, device="cuda").to(dtype)
    y, z = out_mat(3, 40, dtype, 2), out_mat(3, 40, dtype)
    gg.linear(None, 0, None, 40, layout, bias, "relu", None, 0, y, 42, z, 40, 3, 40, 0, dtype, path=path)
    assert torch.equal(y, bias.clamp_min(0).expand(3, 40)) and torch.equal(z, bias.expand(3, 40))
    assert (padding(y) == FILL).all()
    y.fill_(5)
    gg.linear(None, 8, y, 40, layout, bias, "relu", None, 0, y, 40, None, 0, 0, 40, 8, dtype, path=path)
    assert (y == 5).all()
    dw, db = torch.full((8, 40), 3.0, device="cuda"), torch.full((40,), 2.0, device="cuda")
    dw = dw if layout == "kn" else dw.t().contiguous()
    for acc, want in ((True, (3, 2)), (False, (0, 0))):
        gg.linear_backward(None, 40, None, 8, None, 0, layout, None, 0, "none", None, 0, dw, dw.stride(0),
                           db, F32, acc, 0, 40, 8, dtype, path=path)
        assert (dw == want[0]).all() and (db == want[1]).all()
    dx = out_mat(5, 8, dtype)
    gg.linear_backward(None, 0, None, 8, None, 8, layout, None, 0, "none", dx, 8, None, 0, None, F32, False,
                       5, 0, 8, dtype, path=path)
    assert (dx == 0).all()
    status_ok()


@pytest.mark.parametrize("path", ["split", "pair"])
def test_non_finite_values_stay_in_their_rows(path):
    """NaN and infinities of one token reach only that token's row; ragged edges never bring them in."""
    gen = gg_inputs.generator(9)
    M, N, K, dtype = 140, 190, 100, BF16
    x, w = mat(M, K, dtype, gen, ints=True), mat(K, N, dtype, gen, ints=True)
    x.as_strided((M, x.stride(0)), (x.stride(0), 1))[:, K:] = math.nan  # padding beyond K is not read
    clean = (x.double() @ w.double()).to(dtype)
    x[77, 3], x[139, 99] = math.nan, math.inf
    y = out_mat(M, N, dtype)
    call_linear(x, w, "kn", None, "none", None, y, None, path)
    ref = (x.double() @ w.double()).to(dtype)
    keep = torch.ones(M, dtype=torch.bool)
    keep[77] = keep[139] = False
    assert torch.equal(y[keep], clean[keep])
    assert y[77].isnan().all()
    assert torch.equal(y[139].isnan(), ref[139].isnan()) and torch.equal(y[139].isinf(), ref[139].isinf())


# ---- gradients ---------------------------------------------------------------------

def call_backward(dz, x, w, layout, zin, act, dx, dw, db, accumulate, path="auto", **kw):
    import gemm_gather_gb300 as gg
    M, N = dz.shape
    K = x.shape[1]
    gdt = dw.dtype if dw is not None else (db.dtype if db is not None else F32)
    gg.linear_backward(dz, dz.stride(0), x, x.stride(0), w, w.stride(0), layout, zin,
                       zin.stride(0) if zin is not None else 0, act, dx,
                       dx.stride(0) if dx is not None else 0, dw, dw.stride(0) if dw is not None else 0,
                       db, gdt, accumulate, M, N, K, dz.dtype, path=path, **kw)


@pytest.mark.parametrize("path", ["split", "pair"])
@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("grad", ["same", "f32"])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("M,N,K", [(1, 64, 64), (5, 3, 2), (100, 130, 70), (640, 257, 300), (1100, 96, 515)])
def test_integer_gradients_are_exact(M, N, K, accumulate, grad, layout, path):
    gen = gg_inputs.generator(M + N + K)
    dtype = F16 if N % 2 else BF16
    gdt = F32 if grad == "f32" else dtype
    dz, x = mat(M, N, dtype, gen, ints=True), mat(M, K, dtype, gen, ints=True, pad=8)
    w = mat(*((K, N) if layout == "kn" else (N, K)), dtype, gen, ints=True)
    dx = out_mat(M, K, dtype, 3)
    dw, db = out_mat(*w.shape, gdt, 1), torch.full((N,), 1.0, dtype=gdt, device="cuda")
    dw.copy_(gg_inputs.integers(tuple(w.shape), -2, 2, F32, gen))
    dw0, db0 = dw.double(), db.double()
    call_backward(dz, x, w, layout, None, "none", dx, dw, db, accumulate, path)
    assert torch.equal(dx, (dz.double() @ weight64(w, layout).t()).to(dtype))
    g = x.double().t() @ dz.double()
    g = g if layout == "kn" else g.t()
    assert torch.equal(dw, (g + dw0 * accumulate).to(gdt))
    assert torch.equal(db, (dz.double().sum(0) + db0 * accumulate).to(gdt))
    assert (padding(dx) == FILL).all() and (padding(dw) == FILL).all()
    status_ok()


@pytest.mark.parametrize("act", ACTS[1:])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("M,N,K,layout,path", [(19, 300, 260, "kn", "split"), (300, 190, 515, "nk", "pair"),
                                               (300, 190, 515, "kn", "auto")])
def test_input_gradient_through_an_activation(M, N, K, layout, path, dtype, act):
    gen = gg_inputs.generator(3)
    dz = mat(M, N, dtype, gen)
    x = mat(M, K, dtype, gen)
    w = mat(*((K, N) if layout == "kn" else (N, K)), dtype, gen, scale=N ** -0.5)
    zin = mat(M, K, dtype, gen, scale=1.5)
    zin[0, :5] = torch.tensor([0.0, -0.0, 20.0, -20.0, 1e-3])
    dx = out_mat(M, K, dtype)
    call_backward(dz, x, w, layout, zin, act, dx, None, None, False, path)
    p = dz.double() @ weight64(w, layout).t()
    s = slope64(zin.double(), act)  # differences in 64 bits: within 1e-9 of the slope
    err = (N + 4) * 2.0 ** -23 * (dz.double().abs() @ weight64(w, layout).t().abs())
    want = p * s
    bound = SLOPE * err + (2.0 ** -20 + 1e-9) * p.abs() + half_ulp(want, dtype) * 1.01
    assert ((dx.double() - want).abs() <= bound).all()
    z2 = zin.clone()
    call_backward(dz, x, w, layout, z2, act, z2, None, None, False, path)  # dX over z_in
    assert torch.equal(z2, dx)


def test_gradients_against_differences():
    """dX, dW and dbias of sum(G * act(X W + b)) against central differences of that sum in
    float64, at single elements: a wrong formula is off by the size of the gradient, the
    16-bit dZ and results by a few 2^-9 of it."""
    gen = gg_inputs.generator(21)
    M, N, K, dtype = 12, 40, 24, BF16
    x, w = mat(M, K, dtype, gen), mat(K, N, dtype, gen, scale=0.3)
    b, up = torch.randn((N,), generator=gen).to(dtype).cuda(), mat(M, N, dtype, gen)
    import gemm_gather_gb300 as gg
    y, z = out_mat(M, N, dtype), out_mat(M, N, dtype)
    call_linear(x, w, "kn", b, "silu", None, y, z)
    dz = mat(M, N, dtype, gen)
    gg.act_backward(up, up.stride(0), z, z.stride(0), dz, dz.stride(0), "silu", M, N, dtype)
    dx, dw, db = out_mat(M, K, dtype), out_mat(K, N, F32), torch.empty((N,), device="cuda")
    call_backward(dz, x, w, "kn", None, "none", dx, dw, db, False)
    x64, w64, b64, u64 = x.double(), w.double(), b.double(), up.double()

    def total():
        return float((u64 * act64(x64 @ w64 + b64, "silu")).sum())

    for t, g in ((x64, dx), (w64, dw), (b64, db)):
        size = float(g.double().abs().max())
        flat, gf = t.view(-1), g.reshape(-1).double()
        for e in range(0, flat.numel(), max(1, flat.numel() // 17)):
            keep = float(flat[e])
            flat[e] = keep + 1e-4
            up_ = total()
            flat[e] = keep - 1e-4
            down = total()
            flat[e] = keep
            assert abs((up_ - down) / 2e-4 - float(gf[e])) <= 2.0 ** -6 * size


def test_float32_weight_gradient_over_many_tokens():
    """Float32 weight gradients keep float32's precision over long sums: chunks of tokens in
    the tensor core's accumulator (512 of them are within 512 * 2^-23 / 16 truncations of their size),
    added with round-to-nearest; far below the 2^-17 that one long accumulation shows."""
    gen = gg_inputs.generator(2)
    for path in ("split", "pair"):
        M, N, K = 16384, 256, 256
        dz, x = mat(M, N, BF16, gen), mat(M, K, BF16, gen)
        dw = torch.empty((N, K), device="cuda")
        call_backward(dz, x, x, "nk", None, "none", None, dw, None, False, path)
        want = dz.double().t() @ x.double()
        assert float((dw.double() - want).norm() / want.norm()) <= 2.0 ** -19


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("pad", [0, 1, 8])
def test_act_backward(act, dtype, pad):
    import gemm_gather_gb300 as gg
    gen = gg_inputs.generator(4)
    M, N = 37, 1003
    dy, z = mat(M, N, dtype, gen, pad=pad), mat(M, N, dtype, gen, pad=pad, scale=2.0)
    dz = out_mat(M, N, dtype, 5)
    gg.act_backward(dy, dy.stride(0), z, z.stride(0), dz, dz.stride(0), act, M, N, dtype)
    want = dy.double() * slope64(z.double(), act)
    bound = (2.0 ** -20 + 1e-9) * dy.double().abs() + half_ulp(want, dtype) * 1.01
    assert ((dz.double() - want).abs() <= bound).all()
    assert (padding(dz) == FILL).all()
    gg.act_backward(dy, dy.stride(0), z, z.stride(0), dy, dy.stride(0), act, M, N, dtype)  # in place
    assert torch.equal(dy, dz)


# ---- streams, graphs, failure ---------------------------------------------------------

@pytest.mark.parametrize("path", ["split", "pair"])
def test_same_bits_on_another_stream_and_in_a_graph(path):
    gen = gg_inputs.generator(8)
    M, N, K, dtype = 90, 700, 3000, F16
    x, w = mat(M, K, dtype, gen), mat(N, K, dtype, gen, scale=0.02)
    y, y2, y3 = (out_mat(M, N, dtype) for _ in range(3))
    call_linear(x, w, "nk", None, "gelu", None, y, None, path)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call_linear(x, w, "nk", None, "gelu", None, y2, None, path)
        graph = torch.cuda.CUDAGraph()
    side.synchronize()
    with torch.cuda.graph(graph):
        call_linear(x, w, "nk", None, "gelu", None, y3, None, path)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(y, y3)


@pytest.mark.parametrize("path", ["split", "pair"])
def test_a_wait_that_runs_out_is_reported(path):
    """The first stage of one program is never armed: the bounded wait gives up, the status word
    says so, and the same call afterwards is right."""
    import gemm_gather_gb300 as gg
    gen = gg_inputs.generator(8)
    M, N, K, dtype = 300, 300, 1024, F16
    x, w = mat(M, K, dtype, gen, ints=True), mat(K, N, dtype, gen, ints=True)
    y = out_mat(M, N, dtype)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    old = gg.get_wait_limit_ns()
    try:
        gg.set_wait_limit_ns(20_000_000)
        gg.debug_inject_stall(True)
        call_linear(x, w, "kn", None, "none", None, y, None, path, status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == -6
    finally:
        gg.debug_inject_stall(False)
        gg.set_wait_limit_ns(old)
    status.zero_()
    call_linear(x, w, "kn", None, "none", None, y, None, path, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    assert torch.equal(y, (x.double() @ w.double()).to(dtype))


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("M,N,K", [(777, 40, 48), (64, 104, 200), (2048, 240, 248)])
def test_each_reads_what_the_one_before_wrote(M, N, K, graph):
    """Launches that may start under the ones before them: every operand of a call was written by the
    call just before it, and the buffers are overwritten right after the last.  Integers: exact."""
    import gemm_gather_gb300 as gg
    gen = gg_inputs.generator(M + N)

    def ints(r, c):
        return torch.randint(-1, 2, (r, c), generator=gen).to(BF16).cuda()

    dz, x, w, w2 = ints(M, N), ints(M, K), ints(K, N), ints(K, 64)
    dx, dw = (torch.full(s, 99.0, dtype=BF16, device="cuda") for s in ((M, K), (K, N)))
    db, y, y2 = (torch.empty(s, dtype=BF16, device="cuda") for s in ((N,), (M, 64), (M, N)))
    db2 = torch.empty(N, device="cuda")

    def calls():
        gg.linear_backward(dz, N, x, K, w, N, "kn", None, 0, "none", dx, K, dw, N, db, BF16, False, M, N, K, BF16)
        gg.linear(dx, K, w2, 64, "kn", None, "none", None, 0, y, 64, None, 0, M, 64, K, BF16)
        gg.linear(x, K, dw, N, "kn", db, "none", None, 0, y2, N, None, 0, M, N, K, BF16)
        gg.linear_backward(y2, N, None, 0, None, 0, "kn", None, 0, "none", None, 0, None, 0, db2, F32, False, M, N, K,
                           BF16)
        dx.fill_(99.0)
        dw.fill_(99.0)

    if graph:
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            calls()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            calls()
        for out in (y, y2, db, db2):
            out.zero_()
        for _ in range(3):
            g.replay()
    else:
        calls()
    want_dx, want_dw = (dz.double() @ w.double().t()).to(BF16), (x.double().t() @ dz.double()).to(BF16)
    want_db = dz.double().sum(0).to(BF16)
    assert torch.equal(db, want_db)
    assert torch.equal(y, (want_dx.double() @ w2.double()).to(BF16))
    want_y2 = (x.double() @ want_dw.double() + want_db.double()).to(BF16)
    assert torch.equal(y2, want_y2)
    total = want_y2.double().abs().sum(0)  # of whole numbers; float32 is exact below 2^24
    assert (((db2.double() - want_y2.double().sum(0)).abs() == 0) | (total >= 2.0 ** 24)).all()
