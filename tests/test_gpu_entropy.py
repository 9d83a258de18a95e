"""Cross entropy over a vocabulary without stored logits, and its gradients, against float64.

Bounds, from the arithmetic: a logit is a float32 sum over K, off by bz = K 2^-23 sum |x w| (which also
covers an accumulator that truncates); its exponential's argument is a difference times log2 e, (|z - lse| + 1)
2^-22; so lse is off by the largest bz and 2^-20 + |lse| 2^-23, the loss by twice that.  A probability is
off by the factor d = bz + d(lse) + (|z - lse| + 4) 2^-22.  dZ adds its rounding to 16 bits (half a step, and
float16's least step of 2^-24 at a largest weight of 2^13); in the piece whose exponentials
were kept these are off by 2^-12 before, and 0 from 2^-31 of the largest of 32 on; dX and dW are sums of dZ's errors times the other operand, a float32 sum's own bound,
and half an ulp of the output.
"""
import math

import pytest
import torch

import gemm_gather_gb300 as gg
from gemm_gather_gb300 import _lib
from tests import block_oracle as o
from tests.block_oracle import BF16, F16, F32

pytestmark = pytest.mark.gpu


class Case:
    """Inputs, and everything a call writes."""

    def __init__(self, T, V, K, dtype, layout="nk", masked=0.0, seed=0, pad=0, scale=2.5, gdt=None, dx=True, dw=True,
                 weights=None, dirty=True):
        g = torch.Generator().manual_seed(seed + T + 3 * V + 7 * K)
        self.T, self.V, self.K, self.dtype, self.layout = T, V, K, dtype, layout
        self.x = o.put(torch.randn((T, K), generator=g), dtype, 8 * pad)
        w = torch.randn((V, K), generator=g) * scale * max(K, 1) ** -0.5
        self.w = o.put(w if layout == "nk" else w.t(), dtype, 8 * pad)
        self.target = torch.randint(0, V, (T,), generator=g).cuda()
        self.weight = (torch.rand((T,), generator=g) + 0.1).cuda() / T if weights is None else weights.cuda()
        off = torch.rand((T,), generator=g) < masked
        self.weight[off.cuda()] = 0
        if dirty and off.any():      # a masked token's row and target may hold anything
            self.x[off.cuda()] = float("nan")
            self.target[off.cuda()] = 1 << 40
        self.stats, self.loss, self.lse = (torch.full((n,), 7.0, device="cuda") for n in (2, T, T))
        self.dx = o.room(T, K, dtype, pad) if dx else None
        self.dw = o.put(torch.randn(self.w.shape, generator=g), gdt or dtype, pad) if dw else None
        self.before = self.dw.clone() if dw else None

    def call(self, piece=0, accumulate=False, grad_scale=1.0, dx=None, workspace=None, status=None, **kw):
        ld = lambda t: t.stride(0) if t is not None else 0   # noqa: E731
        dx = self.dx if dx is None else dx
        grads = dx is not None or self.dw is not None
        need = gg.linear_cross_entropy_workspace(self.T, self.V, self.K, piece, grads)
        room = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device="cuda") if workspace is None else workspace
        gg.linear_cross_entropy(self.x, ld(self.x), self.w, ld(self.w), self.layout, self.target, self.weight, self.stats,
                                self.loss, self.lse, dx, ld(dx), self.dw, ld(self.dw),
                                self.dw.dtype if self.dw is not None else self.dtype, accumulate, room, self.T, self.V,
                                self.K, self.dtype, piece=piece, grad_scale=grad_scale, status=status, workspace_bytes=need, **kw)
        if workspace is None:
            assert (room[need:] == 0xFF).all()
        return self

    def check(self, accumulate=False, grad_scale=1.0, x=None, dx=None):
        T, V, K, dt = self.T, self.V, self.K, self.dtype
        live = (self.weight != 0) & (self.target >= 0) & (self.target < V)
        x = torch.where(live[:, None], (self.x if x is None else x).double(), 0.0)
        w = self.w.double() if self.layout == "nk" else self.w.double().t()
        tg = torch.where(live, self.target, 0)
        z = x @ w.t()
        lse = torch.logsumexp(z, 1)
        bz = (x.abs() @ w.abs().t()) * (max(K, 1) * 2.0 ** -23)
        dl = bz.amax(1) + 2.0 ** -20 + lse.abs() * 2.0 ** -23
        loss = lse - z.gather(1, tg[:, None])[:, 0]
        tw = torch.where(live, self.weight.double(), 0.0)
        assert (self.lse[~live] == 0).all() and (self.loss[~live] == 0).all()
        assert ((self.lse.double() - lse)[live].abs() <= dl[live]).all()
        assert ((self.loss.double() - loss)[live].abs() <= 2 * dl[live]).all()
        assert abs(float(self.stats[0]) - float((tw * loss).sum())) <= float((tw.abs() * (2 * dl + loss.abs() * 2.0 ** -22)).sum()) + 1e-30
        assert abs(float(self.stats[1]) - float(tw.sum())) <= float(tw.abs().sum()) * 2.0 ** -23 + 1e-30
        p = torch.exp(z - lse[:, None])
        hot = torch.zeros_like(p).scatter_(1, tg[:, None], 1.0)
        coef = (tw * grad_scale)[:, None]
        dz = coef * (p - hot)
        d = bz + dl[:, None] + ((z - lse[:, None]).abs() + 4) * 2.0 ** -22
        half = 2.0 ** (-11 if dt is F16 else -8) + 2.0 ** -12
        least = float(coef.abs().max()) * 2.0 ** -37 if dt is F16 else 0.0
        least = least + coef.abs() * p.amax(1, keepdim=True) * 2.0 ** -31
        err = coef.abs() * (p * torch.expm1(d) + 2.0 ** -23) + dz.abs() * half + least
        dx = self.dx if dx is None else dx
        if dx is not None:
            want = dz @ w
            bound = err @ w.abs() + (dz.abs() @ w.abs()) * (V * 2.0 ** -23) + o.half_ulp(want, dt) * 1.01
            assert ((dx.double() - want).abs() <= bound).all()
            assert (dx[~live] == 0).all()
        if self.dw is not None:
            want = dz.t() @ x
            bound = err.t() @ x.abs() + (dz.abs().t() @ x.abs()) * (T * 2.0 ** -23)
            if accumulate:
                b = self.before.double() if self.layout == "nk" else self.before.double().t()
                want, bound = want + b, bound + b.abs() * 2.0 ** -23
            got = self.dw.double() if self.layout == "nk" else self.dw.double().t()
            assert ((got - want).abs() <= bound + o.half_ulp(want, self.dw.dtype) * 1.01).all()
        for t in (self.dx, self.dw):
            assert t is None or o.untouched(t)
        assert gg.device_status() == 0
        return self


SIZES = [(1, 1, 8), (1, 200, 64), (3, 31, 72), (16, 8192, 512), (27, 1000, 500), (64, 33, 8), (65, 4100, 136), (300, 129, 1000),
         (300, 5000, 264), (777, 2050, 520), (1500, 700, 64)]


@pytest.mark.parametrize("T,V,K", SIZES)
@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_loss_and_gradients(T, V, K, layout, dtype):
    i = SIZES.index((T, V, K))
    masked = (0.0, 0.3, 0.9)[i % 3] if T > 1 else 0.0
    acc = i % 2 == 1
    c = Case(T, V, K, dtype, layout, masked, pad=i % 2, gdt=F32 if i % 4 < 2 else dtype)
    scale = 1024.0 if dtype is F16 else 1.0
    c.call(accumulate=acc, grad_scale=scale).check(acc, scale)


@pytest.mark.parametrize("T,V,K,piece", [(40, 1000, 128, 128), (300, 5000, 264, 1024), (777, 2050, 520, 2048), (130, 300, 72, 256)])
@pytest.mark.parametrize("layout", ["nk", "kn"])
def test_pieces(T, V, K, piece, layout):
    c = Case(T, V, K, BF16, layout, 0.25, gdt=F32)
    c.call(piece).check()
    first = [t.clone() for t in (c.stats, c.loss, c.lse, c.dw, c.dx)]
    c.call(piece)
    for a, b in zip(first, (c.stats, c.loss, c.lse, c.dw, c.dx)):
        assert torch.equal(a, b)                 # the same bits again
    c.call(0).check()
    for a, b in zip(first[:3], (c.stats, c.loss, c.lse)):
        assert torch.equal(a, b)                 # the loss does not depend on the pieces


# dX's contraction goes in shares by the length of a whole piece: the last one, the shortest and first to be
# computed, has fewer blocks of 64 entries than there are shares, which have to come out as zeros
@pytest.mark.parametrize("T,K", [(100, 256), (200, 520)])
@pytest.mark.parametrize("more", [1, 128, 200])
def test_last_piece_shorter_than_the_shares(T, K, more):
    Case(T, 8192 + more, K, BF16, masked=0.25, gdt=F32).call(8192).check()


@pytest.mark.parametrize("T,V,K", [(16, 300, 64), (400, 3000, 520)])
def test_parts_alone(T, V, K):
    c = Case(T, V, K, BF16, masked=0.2).call().check()
    for dx, dw in ((True, False), (False, True), (False, False)):
        d = Case(T, V, K, BF16, masked=0.2, dx=dx, dw=dw).call().check()
        assert torch.equal(c.loss, d.loss) and torch.equal(c.lse, d.lse) and torch.equal(c.stats, d.stats)
    c = Case(T, V, K, BF16, masked=0.2)
    c.stats = c.lse = None
    loss = d.loss.clone()
    c.call()
    assert torch.equal(c.loss, loss)


@pytest.mark.parametrize("T", [5, 700])
def test_every_token_masked(T):
    for acc in (False, True):
        c = Case(T, 500, 136, BF16, masked=2.0, gdt=F32).call(accumulate=acc)
        assert (c.loss == 0).all() and (c.lse == 0).all() and (c.stats == 0).all() and (c.dx == 0).all()
        assert torch.equal(c.dw, c.before) if acc else (c.dw == 0).all()


@pytest.mark.parametrize("keep", [[0], [699], [63, 64], list(range(100, 164)), list(range(0, 700, 7))])
def test_few_tokens_left(keep):
    weights = torch.zeros((700,))
    weights[keep] = torch.linspace(0.5, 1.5, len(keep))
    c = Case(700, 1000, 264, BF16, weights=weights)
    c.x[(weights == 0).cuda()] = float("inf")
    c.call().check()


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("size", [1e-6, 1.0, 3e4, 1e30])
def test_weights_of_any_size(dtype, size):
    """Weights of either sign and of sizes that 16 bits do not hold: the gradient's scale takes them in."""
    if dtype is F16 and size == 1e30:
        scale = 1e-30
    else:
        scale = 1.0 / size
    weights = torch.randn((200,), generator=torch.Generator().manual_seed(1)) * size
    c = Case(200, 600, 136, dtype, weights=weights, gdt=F32)
    c.call(grad_scale=scale).check(grad_scale=float(torch.tensor(scale, dtype=F32)))


@pytest.mark.parametrize("T,V", [(20, 300), (500, 3000)])
def test_large_logits(T, V):
    """Logits of hundreds: exponentials of their differences only."""
    c = Case(T, V, 128, BF16, scale=150.0).call().check()
    assert float(c.lse.max()) > 200


def test_entries_of_probability_zero_and_rows_without_any():
    for T in (4, 300):
        c = Case(T, 400, 8, BF16, dx=False, dw=False)
        c.x[:] = c.x.abs() + 0.1
        c.w[3] = -float("inf")
        c.w[390:] = -float("inf")
        c.target[c.target >= 390] = 5
        c.target[c.target == 3] = 5
        c.target[0] = 395
        c.call()
        z = c.x.double() @ c.w.double().t()
        assert ((c.lse.double() - torch.logsumexp(z, 1)).abs() < 1e-4).all()
        assert c.loss[0] == float("inf") and c.loss[1:].isfinite().all()
        c.w[:] = -float("inf")
        c.call()
        assert c.loss.isnan().all() and (c.lse == -float("inf")).all()
        c = Case(T, 400, 8, BF16)
        c.x[2, 1] = float("nan")
        c.call()
        assert c.loss[2].isnan() and c.loss.isnan().sum() == 1 and c.dx[2].isnan().all() and c.dx.isnan().any(1).sum() == 1


def test_targets_out_of_range_are_masked_and_reported():
    c = Case(70, 300, 72, BF16)
    c.target[5], c.target[69], c.target[30] = -1, 300, 1 << 33
    status = torch.zeros((1,), dtype=torch.int32, device="cuda")
    c.call(status=status).check()
    assert int(status) == _lib.GG_ERR_INVALID_ARG
    c.call()
    assert gg.device_status() == _lib.GG_ERR_INVALID_ARG
    gg.clear_device_status()


@pytest.mark.parametrize("T,V,K", [(33, 200, 64), (600, 2000, 520)])
def test_dx_over_x(T, V, K):
    c = Case(T, V, K, BF16, masked=0.2)
    want = c.call().dx.clone()
    x = c.x.clone()
    c.call(dx=c.x)
    assert torch.equal(c.x, want)
    c.check(x=x, dx=c.x)


def test_outputs_anywhere():
    c = Case(100, 333, 65, F16, gdt=F32)
    c.dx, c.dw = o.room(100, 65, F16, pad=1, shift=1), o.room(333, 65, F32, pad=3, shift=1)
    c.call().check()
    c = Case(100, 333, 65, F16, "kn")
    c.dx, c.dw = o.room(100, 65, F16, pad=1, shift=1), o.room(65, 333, F16, pad=5, shift=3)
    c.call().check()


def test_empty_sizes():
    w = torch.ones((32, 16), dtype=BF16, device="cuda")
    dw, stats = torch.full((32, 16), 3.0, device="cuda"), torch.full((2,), 3.0, device="cuda")
    for acc, want in ((True, 3.0), (False, 0.0)):
        gg.linear_cross_entropy(None, 16, w, 16, "nk", None, None, stats, None, None, None, 16, dw, 16, F32, acc, None, 0, 32,
                                16, BF16)
        assert (dw == want).all() and (stats == 0).all()
    for T in (6, 300):
        c = Case(T, 50, 0, BF16, dx=False, dw=False)
        c.call()
        assert ((c.lse - math.log(50)).abs() < 1e-5).all() and ((c.loss - math.log(50)).abs() < 1e-5).all()


def test_one_entry_is_certain():
    c = Case(90, 1, 64, BF16, gdt=F32).call()
    assert (c.loss == 0).all() and (c.dx == 0).all() and (c.dw == 0).all()


def test_gradients_against_differences():
    """dX and dW against central differences of the loss in float64."""
    c = Case(6, 40, 16, BF16, gdt=F32, masked=0.3, dirty=False).call()
    x, w, tw = c.x.double(), c.w.double(), c.weight.double()

    def f(x, w):
        z = x @ w.t()
        return (tw * (torch.logsumexp(z, 1) - z.gather(1, c.target[:, None])[:, 0])).sum()
    for t, g in ((x, c.dx), (w, c.dw)):
        for i in range(0, t.numel(), 7):
            e = torch.zeros_like(t).view(-1)
            e[i] = 1e-5
            e = e.view(t.shape)
            a = (f(x + e, w) - f(x - e, w)) if t is x else (f(x, w + e) - f(x, w - e))
            slope, got = float(a) / 2e-5, float(g.contiguous().view(-1)[i])
            # dZ's roundings of half a step, its sum's terms of either sign; the output's own
            assert abs(got - slope) <= 2.0 ** -7 * float(tw.max()) * 4


def test_on_another_stream_and_in_a_graph():
    c = Case(500, 3000, 264, BF16, masked=0.3)
    c.call()
    want = [t.clone() for t in (c.stats, c.loss, c.lse, c.dx, c.dw)]
    room = torch.empty((gg.linear_cross_entropy_workspace(500, 3000, 264, 1024),), dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c.call(1024, workspace=room)
    s.synchronize()
    for a, b in zip(want[:3], (c.stats, c.loss, c.lse)):
        assert torch.equal(a, b)
    want = [t.clone() for t in (c.stats, c.loss, c.lse, c.dx, c.dw)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.call(1024, workspace=room)
    # the graph follows what its inputs hold: another mask
    keep = c.weight.clone()
    c.weight[:250] = 0
    for t in (c.stats, c.loss, c.lse, c.dx, c.dw):
        t.zero_()
    g.replay()
    c.check()
    c.weight.copy_(keep)
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, (c.stats, c.loss, c.lse, c.dx, c.dw)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T,V,K", [(16, 2000, 512), (600, 5000, 520)])
def test_a_wait_that_gave_up_is_reported(T, V, K):
    c = Case(T, V, K, BF16)
    status = torch.zeros((1,), dtype=torch.int32, device="cuda")
    gg.set_wait_limit_ns(20_000_000)
    gg.debug_inject_stall(True)
    try:
        c.call(status=status)
        torch.cuda.synchronize()
    finally:
        gg.debug_inject_stall(False)
        gg.set_wait_limit_ns(0)
    assert int(status) == _lib.GG_ERR_TIMEOUT
    status.zero_()
    c.call(status=status).check()
    assert int(status) == 0


def test_many_tokens_and_the_split_of_their_count():
    """More tokens than a block counts at a time (16384), of which every third counts."""
    T = 40000
    weights = torch.zeros((T,))
    weights[1::3] = 1.0 / T
    c = Case(T, 96, 64, BF16, weights=weights, gdt=F32)
    c.call().check()
