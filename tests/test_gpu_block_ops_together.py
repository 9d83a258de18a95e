"""The operators of a step that keeps little, back to back on one stream with one scratch memory, and several calls at
once on streams of their own: the same bits as with a wait after every call."""
import pytest
import torch

import gemm_gather_gb300 as gg
from tests.block_oracle import BF16, F32

pytestmark = pytest.mark.gpu

U8 = torch.uint8


class Step:
    """norm, linear, packing, norm, loss, and back; every call reads what the ones before wrote."""

    def __init__(self, T, D, H, V, seed, act="silu", odd=0):
        g = torch.Generator().manual_seed(seed)
        self.T, self.D, self.H, self.V, self.act = T, D, H, V, act
        r = lambda *s: torch.randn(s, generator=g)                      # noqa: E731
        self.x = r(T, D).to(BF16).cuda()
        self.w1, self.w2 = (r(H, D) * D ** -0.5).to(BF16).cuda(), (r(D, H) * H ** -0.5).to(BF16).cuda()
        self.wv, self.g = (r(V, D) * 2 * D ** -0.5).to(BF16).cuda(), (1 + 0.1 * r(D)).cuda()
        self.target = torch.randint(0, V, (T,), generator=g).cuda()
        self.weight = ((torch.rand((T,), generator=g) < 0.8).float() / T).cuda()
        e = lambda *s, dtype=BF16: torch.empty(s, dtype=dtype, device="cuda")   # noqa: E731
        self.n, self.m, self.h, self.y, self.dh, self.dn = (e(T, D + odd) for _ in range(6))
        self.nc, self.ns, self.zc, self.zs = e(T, D, dtype=U8), e(T, -(-D // 128), dtype=F32), e(T, H, dtype=U8), e(T, -(-H // 128), dtype=F32)
        self.r1, self.r2, self.loss, self.stats = e(T, dtype=F32), e(T, dtype=F32), e(T, dtype=F32), e(2, dtype=F32)
        self.z, self.a, self.dz = e(T, H), e(T, H), e(T, H)
        self.dwv, self.dw1, self.dw2, self.db, self.dg = (e(*s, dtype=F32) for s in ((V, D), (H, D), (D, H), (D,), (D,)))
        self.ws = e(max(gg.linear_cross_entropy_workspace(T, V, D), gg.linear_backward8_workspace(T, max(D, H)),
                        gg.rms_norm_backward_workspace(T, D)), dtype=U8)

    def calls(self):
        s, T, D, H, V = self, self.T, self.D, self.H, self.V
        yield lambda: gg.rms_norm(s.x, D, None, 0, s.g, 1e-6, None, 0, s.n, D, s.nc, D, s.ns, s.ns.stride(0), s.r1, T, D, BF16)
        yield lambda: gg.linear(s.n, D, s.w1, D, "nk", None, s.act, None, 0, s.a, H, s.z, H, T, H, D, BF16)
        yield lambda: gg.pack8(s.z, H, s.zc, H, s.zs, s.zs.stride(0), T, H, BF16)
        yield lambda: gg.unpack8(s.zc, H, s.zs, s.zs.stride(0), s.act, s.a, H, T, H, BF16)
        yield lambda: gg.linear(s.a, H, s.w2, H, "nk", None, "none", None, 0, s.m, D, None, 0, T, D, H, BF16)
        o = s.h.stride(0)
        yield lambda: gg.rms_norm(s.m, D, s.x, D, s.g, 1e-6, s.h, o, s.y, D, None, 0, None, 0, s.r2, T, D, BF16)
        yield lambda: gg.linear_cross_entropy(s.y, D, s.wv, D, "nk", s.target, s.weight, s.stats, s.loss, None, s.y, D, s.dwv, D,
                                              F32, False, s.ws, T, V, D, BF16)
        yield lambda: gg.rms_norm_backward(s.y, D, s.h, o, s.r2, s.g, None, 0, s.dh, D, s.dg, F32, False, s.ws, T, D, BF16)
        yield lambda: gg.linear_backward8(s.dh, D, s.zc, H, s.zs, s.zs.stride(0), s.act, s.w2, H, "nk", s.dz, H, s.dw2, H, s.db,
                                          F32, False, s.ws, T, D, H, BF16)
        yield lambda: gg.linear_backward8(s.dz, H, s.nc, D, s.ns, s.ns.stride(0), "none", s.w1, D, "nk", s.dn, D, s.dw1, D, None,
                                          F32, False, s.ws, T, H, D, BF16)
        yield lambda: gg.rms_norm_backward(s.dn, D, s.x, D, s.r1, s.g, s.dh, D, s.dn, D, s.dg, F32, True, s.ws, T, D, BF16)
        # on to the next round: what this one left changes its inputs
        yield lambda: gg.rms_norm(s.dn, D, s.x, D, s.g, 1e-6, None, 0, s.x, D, None, 0, None, 0, None, T, D, BF16)

    def run(self, rounds, wait):
        for _ in range(rounds):
            for call in self.calls():
                call()
                if wait:
                    torch.cuda.synchronize()

    def outputs(self):
        return [self.x, self.nc, self.ns, self.zc, self.zs, self.r1, self.r2, self.loss, self.stats, self.dwv, self.dw1, self.dw2,
                self.db, self.dg, self.dz]


SIZES = [(40, 256, 512, 1000, 0), (300, 264, 520, 3000, 0), (700, 512, 1024, 5000, 0), (700, 512, 1024, 5000, 1),
         (1300, 1024, 512, 2000, 0)]


def same(a, b):
    return all(torch.equal(p.view(U8) if p.dtype == U8 else p, q.view(U8) if q.dtype == U8 else q)
               for p, q in zip(a.outputs(), b.outputs()))


@pytest.mark.parametrize("T,D,H,V,odd", SIZES)
@pytest.mark.parametrize("act", ["silu", "relu"])
def test_back_to_back(T, D, H, V, odd, act):
    a, b = (Step(T, D, H, V, 7, act, odd) for _ in range(2))
    a.run(4, wait=True)
    b.run(4, wait=False)
    torch.cuda.synchronize()
    assert same(a, b) and a.loss.isfinite().all() and a.dw1.isfinite().all() and gg.device_status() == 0


def test_at_once_on_streams_of_their_own():
    sizes = [(300, 264, 520, 3000), (700, 512, 1024, 5000), (40, 256, 512, 1000)]
    alone = [Step(*s, seed=k) for k, s in enumerate(sizes)]
    for a in alone:
        a.run(3, wait=True)
    together = [Step(*s, seed=k) for k, s in enumerate(sizes)]
    streams = [torch.cuda.Stream() for _ in sizes]
    torch.cuda.synchronize()
    for _ in range(3):
        calls = [list(t.calls()) for t in together]
        for k in range(len(calls[0])):
            for c, st in zip(calls, streams):
                with torch.cuda.stream(st):
                    c[k]()
    torch.cuda.synchronize()
    assert all(same(a, b) for a, b in zip(alone, together)) and gg.device_status() == 0


def test_graphs_at_once():
    """Two graphs with scratch memory of their own, replayed side by side."""
    sizes = [(300, 264, 520, 3000), (700, 512, 1024, 5000)]
    alone, captured = ([Step(*s, seed=k) for k, s in enumerate(sizes)] for _ in range(2))
    for a in alone:
        a.run(3, wait=True)
    Step(*sizes[0], seed=9).run(1, wait=True)          # (every kernel set up before a capture)
    graphs, streams = [], [torch.cuda.Stream() for _ in sizes]
    for c in captured:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run(1, wait=False)
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(3):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    assert all(same(a, b) for a, b in zip(alone, captured)) and gg.device_status() == 0
