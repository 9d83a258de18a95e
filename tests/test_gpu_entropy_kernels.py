"""Every kernel that the vocabulary's cross entropy chooses between by its sizes, each named from what a call
launches: logits in one chunk and in several, on CTA pairs and split; the kept exponentials; the gradients' products
with sums over tokens in one chunk and in several, together and alone.  Values are held to test_gpu_entropy.py's
bounds, and the losses to the closer one of entropy_oracle.py."""
import pytest
import torch

import gemm_gather_gb300 as gg
from tests import entropy_oracle as e
from tests.block_oracle import BF16, F16, F32
from tests.launched import variants
from tests.test_gpu_entropy import Case

pytestmark = pytest.mark.gpu

LSE, SOFT, VOCAB, LSE_SHORT = 4, 5, 6, 9      # the products' epilogues, as the kernels number them
ONE_CHUNK, CHUNK = 1792, 1024                                  # logits of longer contractions come in chunks


def products(c, **kw):
    """(kernel, epilogue, second epilogue) of the call's products, in order, and how often it finishes kept
    exponentials."""
    room = torch.empty((1 << 28,), dtype=torch.uint8, device="cuda")

    def call():
        c.call(workspace=room, **kw)
    call()
    all_ = variants(call, "split_kernel", "pair_kernel", "kept_kernel")
    found = [(k[:-7], n[0], n[1] if k == "pair_kernel" else -1) for k, n, _ in all_ if k != "kept_kernel"]
    return found, len(all_) - len(found)


def check_losses(c, chunk):
    live = c.weight != 0
    w = c.w if c.layout == "nk" else c.w.t()
    want, lse = e.losses64(c.x[live], w, c.target[live])
    assert e.relative(c.loss[live], want) <= e.loss_bound(chunk)
    assert e.relative(c.lse[live], lse) <= e.loss_bound(chunk)


@pytest.mark.parametrize("T,V,K,piece", [(600, 700, 1800, 0), (600, 300, 2100, 0), (600, 3000, 2000, 2048), (600, 3000, 3584, 2048)])
@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_logits_in_chunks(T, V, K, piece, layout, dtype):
    scale = 1024.0 if dtype is F16 else 1.0
    c = Case(T, V, K, dtype, layout, 0.25, gdt=F32 if K % 400 == 0 else dtype)
    c.call(piece, grad_scale=scale).check(grad_scale=scale)
    check_losses(c, CHUNK)
    found, kept = products(c, piece=piece, grad_scale=scale)
    assert found[0] == ("pair", LSE, -1) and kept == 1


@pytest.mark.parametrize("T,V,K", [(600, 700, 520), (600, 3000, 1000), (600, 3000, 1792)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_logits_in_one_chunk(T, V, K, dtype):
    c = Case(T, V, K, dtype, "nk", 0.25)
    c.call().check()
    check_losses(c, K)
    found, kept = products(c)
    assert found[0] == ("pair", LSE_SHORT, -1) and kept == 1


@pytest.mark.parametrize("K", [520, 2100])
@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_few_tokens(K, layout, dtype):
    c = Case(40, 300, K, dtype, layout, 0.25)
    c.call().check()
    check_losses(c, K if K <= ONE_CHUNK else CHUNK)
    found, kept = products(c)
    assert found[0] == ("split", LSE, -1) and kept == 0


@pytest.mark.parametrize("T,V,K", [(600, 3000, 264), (2000, 500, 64)])
def test_short_logits_are_multiplied_twice(T, V, K):
    c = Case(T, V, K, BF16, masked=0.25)
    c.call().check()
    check_losses(c, K)
    found, kept = products(c)
    assert kept == 0 and any(f[1] == SOFT for f in found)


@pytest.mark.parametrize("gdt", [F32, BF16])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("dx", [True, False])
def test_weight_gradients_of_many_tokens(gdt, accumulate, dx):
    """More than 16384 tokens: sums in chunks, whatever the gradient's type."""
    c = Case(17000, 96, 64, BF16, masked=0.05, gdt=gdt, dx=dx)
    c.call(accumulate=accumulate).check(accumulate)
    found, _ = products(c, accumulate=accumulate)
    last = found[-1]
    assert (last[2] if last[2] >= 0 else last[1]) == VOCAB


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("layout", ["nk", "kn"])
def test_float32_weight_gradients_over_chunks_of_tokens(layout, accumulate):
    """2000 tokens: float32 weight gradients are sums of chunks of 896."""
    c = Case(2000, 700, 264, BF16, layout, 0.1, gdt=F32)
    c.call(accumulate=accumulate).check(accumulate)
    found, _ = products(c, accumulate=accumulate)
    last = found[-1]
    assert (last[2] if last[2] >= 0 else last[1]) == VOCAB


@pytest.mark.parametrize("T,V,K", [(600, 3000, 520), (600, 700, 2100)])
def test_large_logits_and_kept_exponentials(T, V, K):
    c = Case(T, V, K, BF16, scale=150.0).call().check()
    assert float(c.lse.max()) > 200
    assert products(c)[1] == 1


@pytest.mark.parametrize("T,V,K", [(100, 8192, 256), (64, 16000, 256), (300, 2000, 512)])
def test_a_pair_for_every_share_of_dx(T, V, K):
    """Where few tiles are left to the pairs, the shares of dX's contraction are tiles too."""
    c = Case(T, V, K, BF16)
    room = torch.zeros((gg.linear_cross_entropy_workspace(T, V, K),), dtype=torch.uint8, device="cuda")

    def call():
        c.call(workspace=room)
    call()
    c.check()
    shares = int(room[:12].view(torch.int32)[2])                   # as the device decided
    kernel, numbers, grid = variants(call, "pair_kernel")[-1]
    assert numbers[0] == VOCAB and numbers[1] >= 0 and shares > 1
    most = numbers[2]                                              # tokens (dX) and entries (dW) of a tile, at most
    tiles = -(-K // 256) * -(-T // most) * shares + -(-K // 256) * -(-V // most)
    assert grid[0] // 2 >= min(76, tiles)
