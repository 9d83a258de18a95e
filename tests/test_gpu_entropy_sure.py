"""Tokens that the vocabulary's loss is sure of, and logits of any size, against float64.

Hidden states are rows of the unit matrix, so that a token's logits are a column of W, exactly: no product is
rounded, and what is off is the softmax alone.  A term of the sum of exponentials is off by its argument's rounding
and log2 e's (the argument times 2^-23) and by three exponentials on its way (of its 32 entries' largest logit, of
the tile's, of all: 2^-22 each); a sum of up to 700 entries rounds 32 times (16 in a thread, 1, 5, and at most 10
partial sums that are not 0): 2^-24 each.  So a loss is off by 44 2^-24, the mean argument times 2^-23, and its own
logarithm's and sum's rounding, 2^-22 of it, whatever the logits' size.  lse is rounded to its own size.
"""
import pytest
import torch

from tests.block_oracle import BF16, F16, F32
from tests.test_gpu_entropy import Case

pytestmark = pytest.mark.gpu


# T, V, K: pairs without and with kept exponentials, and with logits in chunks
PAIRS = [(600, 700, 64), (600, 700, 512), (600, 300, 2112)]


def exact_logits(T, V, K, dtype, logits, layout="nk", **kw):
    """A case whose token t has the logits of column t mod K of ``logits``, a V x K matrix."""
    c = Case(T, V, K, dtype, layout, gdt=F32, **kw)
    c.x[:] = torch.eye(K, device="cuda").to(dtype).repeat(-(-T // K), 1)[:T]
    c.w.copy_((logits if layout == "nk" else logits.t()).to(dtype))
    return c


def check_losses(c):
    w = c.w.double() if c.layout == "nk" else c.w.double().t()
    z = w.t()[torch.arange(c.T, device="cuda") % c.K]
    top = z.amax(1)
    below = top[:, None] - z
    rest = torch.log(torch.exp(-below).sum(1))
    mean = (torch.exp(-below - rest[:, None]) * below).sum(1)
    tol = (44 + 2 * mean) * 2.0 ** -24
    loss = top - z.gather(1, c.target[:, None])[:, 0] + rest
    assert ((c.loss.double() - loss).abs() <= tol + loss * 2.0 ** -22).all()
    assert ((c.lse.double() - top - rest).abs() <= tol + rest * 2.0 ** -22 + c.lse.double().abs() * 2.0 ** -24).all()


def sure(T, V, K, dtype, layout="nk", **kw):
    """Targets are the largest logit, 100 to 250, and 2 to 12 above the others: probabilities up to 1 - 0.002."""
    g = torch.Generator().manual_seed(T + K)
    top = 100 + torch.randint(0, 151, (K,), generator=g).float()
    gap = 2 + torch.randint(0, 11, (K,), generator=g).float()
    logits = top - gap - torch.randint(0, 5, (V, K), generator=g)
    a = torch.randint(0, V, (K,), generator=g)
    logits[a, torch.arange(K)] = top
    c = exact_logits(T, V, K, dtype, logits.cuda(), layout, **kw)
    c.target = a[torch.arange(T) % K].cuda()
    return c


def huge(T, V, K, layout="nk", **kw):
    """Two entries share the largest logit, of 2^33 to 2^40 and either sign; the others are far below."""
    g = torch.Generator().manual_seed(T + K)
    size = torch.exp2(33 + 7 * torch.rand((K,), generator=g)).to(BF16).float()
    size = torch.where(torch.rand((K,), generator=g) < 0.5, size, -size)
    logits = (size - size.abs() * (0.1 + torch.rand((V, K), generator=g))).to(BF16)
    a = torch.randint(0, V, (K,), generator=g)
    b = (a + 1 + torch.randint(0, V - 1, (K,), generator=g)) % V
    k = torch.arange(K)
    logits[a, k] = logits[b, k] = size.to(BF16)
    c = exact_logits(T, V, K, BF16, logits.cuda(), layout, **kw)
    c.target = torch.where(torch.rand((T,), generator=g) < 0.5, a[torch.arange(T) % K], b[torch.arange(T) % K]).cuda()
    return c


@pytest.mark.parametrize("layout", ["nk", "kn"])
def test_losses_of_few_tokens(layout):
    for c in (sure(40, 300, 64, BF16, layout), sure(40, 300, 64, F16, layout), huge(40, 300, 64, layout)):
        check_losses(c.call())


@pytest.mark.parametrize("T,V,K", PAIRS)
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("gradients", [False, True])
def test_losses_on_pairs(T, V, K, dtype, gradients):
    check_losses(sure(T, V, K, dtype, dx=gradients, dw=gradients).call())
    if dtype is BF16:
        check_losses(huge(T, V, K, dx=gradients, dw=gradients).call())


def check_gradients(c):
    """dW's columns: sums of the gradients of their tokens' logits.

    A probability is off by what the sum of exponentials is, its own argument and exponential, and two roundings;
    1 is taken from a target's with one more.  Then half a step of 16 bits, before that of an exponential that was
    kept (2^-12, nothing below 2^-31 of the largest; the largest is 1, exactly), and a truncating sum of the tokens that
    are not 0."""
    w = c.w.double() if c.layout == "nk" else c.w.double().t()
    k = torch.arange(c.T, device="cuda") % c.K
    z = w.t()[k]
    below = z.amax(1, keepdim=True) - z
    e = torch.exp(-below)
    total = e.sum(1, keepdim=True)
    p = e / total
    mean = (p * below).sum(1, keepdim=True)
    hot = torch.zeros_like(p).scatter_(1, c.target[:, None], 1.0)
    coef = c.weight.double()[:, None]
    others = torch.where(hot > 0, 0.0, e).sum(1, keepdim=True)       # 1 - p of a target without the cancellation
    dz = coef * torch.where(hot > 0, -others / total, p)
    err = coef * p * ((48 + 2 * mean) * 2.0 ** -24 + below * 2.0 ** -23 + 2.0 ** -22) + coef * hot * 2.0 ** -23
    err = err + coef * torch.where(below == 0, 0.0, p) * 2.0 ** -12 + coef * p.amax(1, keepdim=True) * 2.0 ** -31
    err = (err + dz.abs() * 2.0 ** (-11 if c.dtype is F16 else -8)) + (float(coef.max()) * 2.0 ** -37 if c.dtype is F16 else 0)
    got = c.dw.double() if c.layout == "nk" else c.dw.double().t()
    want, bound = torch.zeros_like(got), torch.zeros_like(got)
    want.index_add_(1, k, dz.t())
    bound.index_add_(1, k, (err + dz.abs() * (-(-c.T // c.K) * 2.0 ** -23)).t())
    assert ((got - want).abs() <= bound).all()


@pytest.mark.parametrize("T,V,K", [(40, 300, 64)] + PAIRS)
@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("piece", [0, 128])
def test_gradients(T, V, K, layout, piece):
    for c in (sure(T, V, K, F16, layout), sure(T, V, K, BF16, layout), huge(T, V, K, layout)):
        check_gradients(c.call(piece))


@pytest.mark.parametrize("layout", ["nk", "kn"])
def test_the_targets_gradient_does_not_depend_on_the_pieces(layout):
    """Confident tokens with logits of about 110 from a long contraction, whose sums differ by 2e-6 of that when they are
    summed in one chunk and in several: as much as 2 % of 1 - p.  A target's row of dW is its token's term, the same
    in every piece, and the others' probabilities, each off by a logit of one chunk (5.5e-10 K 115 <= 2^-12 of it) or a
    kept exponential (2^-12), and half a step of 2^-11 either way: 3 2^-11 between the two.  float32 sums: 2^-20."""
    T, V, K = 600, 1500, 3584
    g = torch.Generator().manual_seed(1)
    x = torch.randn((T, K), generator=g)
    x[:, :64] = 1
    w = torch.randn((V, K), generator=g) * 0.5 * K ** -0.5
    w[:, :64] = 100 / 64
    target = torch.randperm(V, generator=g)[:T]
    w[target, 64:] += x[:, 64:] * (11.5 / x[:, 64:].square().sum(1, keepdim=True))
    c = Case(T, V, K, F16, layout, gdt=F32)
    c.x.copy_(x.to(F16)), c.w.copy_((w if layout == "nk" else w.t()).to(F16))
    c.target = target.cuda()
    rows = []
    for piece in (0, 128):
        c.call(piece)
        rows.append((c.dw if layout == "nk" else c.dw.t())[c.target].double())
    x64 = c.x.double()
    w64 = c.w.double() if layout == "nk" else c.w.double().t()
    p = torch.softmax(x64 @ w64.t(), 1)[:, c.target]
    rest = 1 - p.diagonal()
    assert float(rest.median()) < 0.02 and float((x64 @ w64.t()).max()) < 115
    others = c.weight.double()[:, None] * p
    others.fill_diagonal_(0)
    own = (c.weight.double() * rest)[:, None] * x64.abs()
    bound = (others.t() @ x64.abs()) * 3 * 2.0 ** -11 + (others.t() @ x64.abs() + own) * 2.0 ** -20
    assert ((rows[0] - rows[1]).abs() <= bound).all()
