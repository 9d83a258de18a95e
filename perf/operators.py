"""The operators of one training or serving step next to the gathered matmul: cases, plain forms, exact values.

A weight is held as row blocks by the ranks of a symmetric heap and gathered; a linear layer applies it
(bias, activation, residual), a clipped policy loss turns the logits into a loss and their gradient, the
layer's backward pass turns that into weight gradients, and AdamW updates each rank's row block.  Three
operators are listed here: ``linear`` (forward and backward), ``policy_loss`` and ``adamw``.

With ``own`` false, ``run`` computes them in their plain form: elementary torch operations in float32,
rounded once at the end.  With ``own`` true it calls the library.  ``exact`` gives the same outputs from
the definitions in float64.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
STATE_BLOCK = 256          # elements that share one scale of the 8-bit optimizer states
MASK32 = 0xFFFFFFFF


# --------------------------------------------------------------------------- #
# Cases                                                                       #
# --------------------------------------------------------------------------- #

def listed():
    return [
        # one token through a layer of the benchmark's K x N, weight rows gathered (N x K): decoding
        dict(name="linear 1 token", op="linear", M=1, N=3584, K=8192, dtype="bf16", layout="nk",
             bias=True, act="silu", residual=False, z=False),
        # a small ragged batch of decoding requests, odd sizes, the matmul's own K x N layout
        dict(name="linear 27 tokens odd", op="linear", M=27, N=1531, K=2011, dtype="f16", layout="kn",
             bias=True, act="none", residual=True, z=False),
        # a prompt (the benchmark's M_local=1024 product), everything the epilogue does, Z kept for training
        dict(name="linear 1024 full", op="linear", M=1024, N=3584, K=8192, dtype="f16", layout="kn",
             bias=True, act="gelu", residual=True, z=True),
        # a training batch at the largest M_local
        dict(name="linear 16384", op="linear", M=16384, N=3584, K=8192, dtype="bf16", layout="nk",
             bias=True, act="gelu_tanh", residual=False, z=True),
        # gradients of a small layer over a ragged batch, 16-bit gradients
        dict(name="backward 777 odd", op="backward", M=777, N=1000, K=1523, dtype="bf16", layout="kn",
             act="silu", grad="bf16", accumulate=False),
        # gradients of the benchmark's layer, accumulated in f32 over the data shards
        dict(name="backward 4096 f32 acc", op="backward", M=4096, N=3584, K=8192, dtype="bf16", layout="nk",
             act="gelu", grad="f32", accumulate=True),
        # a few generated tokens scored against a small vocabulary
        dict(name="loss 16 x 8192", op="loss", T=16, V=8192, dtype="bf16", masked=0.0, kl=True, old=True,
             inplace=False),
        # a training batch of tokens with prompt tokens masked out, odd vocabulary
        dict(name="loss 4096 x 100003", op="loss", T=4096, V=100003, dtype="bf16", masked=0.25, kl=True,
             old=True, inplace=True),
        # float32 logits, first update of a batch (the old policy is the present one)
        dict(name="loss 8191 x 32768 f32", op="loss", T=8191, V=32768, dtype="f32", masked=0.1, kl=False,
             old=False, inplace=False),
        # many small tensors: biases and norms of a model; launch count is what matters
        dict(name="adamw 200 small", op="adamw", tensors=200, least=17, most=8192, param="f32", grad="f32",
             state=32, copy=None),
        # one rank's row block of the benchmark's weights, f32 masters with the 16-bit copy that is gathered
        dict(name="adamw 117M f32 states", op="adamw", tensors=4, least=3584 * 8192, most=3584 * 8192,
             param="f32", grad="bf16", state=32, copy="bf16"),
        # the same with states in 8 bits
        dict(name="adamw 117M 8-bit states", op="adamw", tensors=4, least=3584 * 8192, most=3584 * 8192,
             param="f32", grad="bf16", state=8, copy="bf16"),
    ]


def _log_int(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["linear", "linear", "backward", "loss", "adamw", "adamw"])
    if op == "linear":
        return dict(op=op, M=_log_int(rng, 1, 16384), N=_log_int(rng, 64, 3584), K=_log_int(rng, 64, 8192),
                    dtype=rng.choice(["f16", "bf16"]), layout=rng.choice(["kn", "nk"]),
                    bias=rng.random() < 0.7, act=rng.choice(ACTS), residual=rng.random() < 0.5,
                    z=rng.random() < 0.5)
    if op == "backward":
        return dict(op=op, M=_log_int(rng, 16, 4096), N=_log_int(rng, 64, 3584), K=_log_int(rng, 64, 8192),
                    dtype=rng.choice(["f16", "bf16"]), layout=rng.choice(["kn", "nk"]),
                    act=rng.choice(ACTS), grad=rng.choice(["same", "f32"]), accumulate=rng.random() < 0.5)
    if op == "loss":
        V = _log_int(rng, 64, 100003)
        T = _log_int(rng, 1, min(16384, 4096 * 100003 // V))
        return dict(op=op, T=T, V=V, dtype=rng.choice(["f16", "bf16", "f32"]),
                    masked=rng.choice([0.0, 0.3, 0.9]) if T >= 64 else 0.0,
                    kl=rng.random() < 0.7, old=rng.random() < 0.7, inplace=rng.random() < 0.3)
    most = _log_int(rng, 256, 4 << 20)
    param = rng.choice(["f32", "f32", "bf16", "f16"])
    return dict(op=op, tensors=_log_int(rng, 1, 24), least=max(1, most // rng.choice([1, 4, 64])), most=most,
                param=param, grad=rng.choice(["f32", "bf16", "f16"]), state=rng.choice([32, 8]),
                copy=rng.choice([None, "bf16", "f16"]) if param == "f32" else None)


# --------------------------------------------------------------------------- #
# Inputs                                                                      #
# --------------------------------------------------------------------------- #

def _pitch(n):
    """Row pitch of a matrix the tensor maps read: whole 16-byte units."""
    return (n + 7) // 8 * 8


def _matrix(rows, cols, dtype, g, scale=1.0):
    """rows x cols normal values, a view of rows that start on 16-byte boundaries."""
    buf = torch.empty((rows, _pitch(cols)), dtype=dtype, device="cuda")
    step = max(1, (1 << 26) // max(1, _pitch(cols)))
    for r in range(0, rows, step):
        part = torch.randn((min(step, rows - r), _pitch(cols)), generator=g, device="cuda")
        buf[r:r + step] = (part * scale).to(dtype)
    return buf[:, :cols]


def _adamw_sizes(case):
    lo, hi, n = case["least"], case["most"], case["tensors"]
    if n == 1 or lo == hi:
        return [hi] * n
    return [int(round(lo * (hi / lo) ** (i / (n - 1)))) for i in range(n)]


def _places(sizes):
    """(first element, first scale, elements) of each tensor in the flat buffers."""
    at, first, places = 0, 0, []
    for n in sizes:
        places.append((at, first, n))
        at, first = at + _pitch(n), first - (-n // STATE_BLOCK)
    return places


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * int(seed) + 17)
    s = {"case": case}
    if case["op"] in ("linear", "backward"):
        M, N, K, dt = case["M"], case["N"], case["K"], DT[case["dtype"]]
        s["x"] = _matrix(M, K, dt, g)
        s["w"] = _matrix(*((K, N) if case["layout"] == "kn" else (N, K)), dt, g, K ** -0.5)
    if case["op"] == "linear":
        s["bias"] = _matrix(1, N, dt, g, 0.5)[0] if case["bias"] else None
        s["residual"] = _matrix(M, N, dt, g) if case["residual"] else None
        s["y"] = torch.empty((M, _pitch(N)), dtype=dt, device="cuda")[:, :N]
        s["z"] = torch.empty((M, _pitch(N)), dtype=dt, device="cuda")[:, :N] if case["z"] else None
    elif case["op"] == "backward":
        gdt = dt if case["grad"] in ("same", case["dtype"]) else torch.float32
        s["dz"] = _matrix(M, N, dt, g, 0.25)
        s["zin"] = _matrix(M, K, dt, g) if case["act"] != "none" else None
        s["dx"] = torch.empty((M, _pitch(K)), dtype=dt, device="cuda")[:, :K]
        s["dw"] = torch.randn(s["w"].shape, generator=g, device="cuda").to(gdt)
        s["db"] = torch.randn((N,), generator=g, device="cuda").to(gdt)
    elif case["op"] == "loss":
        T, V, dt = case["T"], case["V"], DT[case["dtype"]]
        s["logits"] = _matrix(T, V, dt, g, 2.5)
        s["target"] = torch.randint(0, V, (T,), generator=g, device="cuda")
        # what a sampler saw: the present policy's log probability, a little earlier
        logp = torch.cat([torch.log_softmax(s["logits"][r:r + 512].float(), 1).gather(
            1, s["target"][r:r + 512, None])[:, 0] for r in range(0, T, 512)])
        rnd = torch.randn((3, T), generator=g, device="cuda")
        s["old"] = logp + 0.2 * rnd[0] if case["old"] else None
        s["ref"] = logp + 0.5 * rnd[1] if case["kl"] else None
        s["adv"] = rnd[2].contiguous()
        keep = torch.rand((T,), generator=g, device="cuda") >= case["masked"]
        s["weight"] = keep.float() / max(1.0, float(keep.sum()))
        s["grad"] = s["logits"] if case["inplace"] else torch.empty((T, _pitch(V)), dtype=dt, device="cuda")[:, :V]
        s["logp"] = torch.empty((T,), device="cuda")
        s["stats"] = torch.empty((4,), device="cuda")
        s["hyper"] = dict(inv_temperature=1.0, clip_low=0.2, clip_high=0.28,
                          kl_coef=0.04 if case["kl"] else 0.0,
                          grad_scale=1024.0 if case["dtype"] == "f16" else 1.0)
    else:
        # one flat buffer of each kind, as a sharded optimizer keeps them; tensors start on 16-byte boundaries
        sizes = _adamw_sizes(case)
        total = sum(_pitch(n) for n in sizes)
        flat = {"param": (0.02 * torch.randn((total,), generator=g, device="cuda")).to(DT[case["param"]]),
                "grad": (1e-2 * torch.randn((total,), generator=g, device="cuda")).to(DT[case["grad"]])}
        m, v = 3e-3 * torch.randn((total,), generator=g, device="cuda"), 1e-4 * torch.rand((total,), generator=g, device="cuda")
        if case["state"] == 8:
            for k in ("m", "v"):
                flat[k] = torch.zeros((total,), dtype=torch.float8_e4m3fn, device="cuda")
                flat[k + "_scale"] = torch.zeros((sum(-(-n // STATE_BLOCK) for n in sizes),), device="cuda")
        else:
            flat["m"], flat["v"] = m, v
        if case["copy"]:
            flat["copy"] = torch.zeros((total,), dtype=DT[case["copy"]], device="cuda")
        s["flat"], s["tensors"] = flat, []
        for at, first, n in _places(sizes):
            t = {k: f[first:first - (-n // STATE_BLOCK)] if k.endswith("_scale") else f[at:at + n] for k, f in flat.items()}
            if case["state"] == 8:
                for k, x in (("m", m[at:at + n]), ("v", v[at:at + n].sqrt())):
                    code, scale = _to_codes(x, None)
                    t[k].copy_(code)
                    t[k + "_scale"].copy_(scale)
            s["tensors"].append(t)
        s["grad_scale"] = torch.full((1,), 0.5, device="cuda")
        s["hyper"] = dict(lr=3e-4, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1)
        s["step"], s["seed"] = 100, 12345
    return s


# --------------------------------------------------------------------------- #
# One pass                                                                    #
# --------------------------------------------------------------------------- #

def run(state):
    op = state["case"]["op"]
    if own:
        return {"linear": _own_linear, "backward": _own_backward, "loss": _own_loss, "adamw": _own_adamw}[op](state)
    return {"linear": _plain_linear, "backward": _plain_backward, "loss": _plain_loss, "adamw": _plain_adamw}[op](state)


def _own_linear(s):
    import gemm_gather_gb300 as gg
    c, z, r = s["case"], s["z"], s["residual"]
    gg.linear(s["x"], s["x"].stride(0), s["w"], s["w"].stride(0), c["layout"], s["bias"], c["act"],
              r, r.stride(0) if r is not None else 0, s["y"], s["y"].stride(0),
              z, z.stride(0) if z is not None else 0, c["M"], c["N"], c["K"], s["x"].dtype)
    return [s["y"]] if z is None else [s["y"], z]


def _own_backward(s):
    import gemm_gather_gb300 as gg
    c, zin = s["case"], s["zin"]
    gg.linear_backward(s["dz"], s["dz"].stride(0), s["x"], s["x"].stride(0), s["w"], s["w"].stride(0),
                       c["layout"], zin, zin.stride(0) if zin is not None else 0, c["act"],
                       s["dx"], s["dx"].stride(0), s["dw"], s["dw"].stride(0), s["db"], s["dw"].dtype,
                       c["accumulate"], c["M"], c["N"], c["K"], s["x"].dtype)
    return [s["dx"], s["dw"], s["db"]]


def _own_loss(s):
    import gemm_gather_gb300 as gg
    c, h = s["case"], s["hyper"]
    gg.policy_loss(s["logits"], s["logits"].stride(0), s["target"], s["old"], s["ref"], s["adv"], s["weight"],
                   c["T"], c["V"], s["logits"].dtype, s["stats"], s["logp"], s["grad"], s["grad"].stride(0), **h)
    return [s["stats"], s["logp"], s["grad"]]


def _own_adamw(s):
    import gemm_gather_gb300 as gg
    if "table" not in s:  # a program describes its tensors once, before its first step
        s["table"] = gg.adamw_tensors(s["tensors"], state_bits=s["case"]["state"])
    gg.adamw(s["table"], s["step"], grad_scale=s["grad_scale"], seed=s["seed"], **s["hyper"])
    s["step"] += 1
    return _adamw_outputs(s)


def _act(z, act):
    if act == "none":
        return z
    if act == "relu":
        return torch.clamp_min(z, 0)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * 0.7071067811865476))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(0.7978845608028654 * (z + 0.044715 * z * z * z)))
    return z / (1 + torch.exp(-z))


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * 0.7071067811865476)) + z * torch.exp(-0.5 * z * z) * 0.3989422804014327
    if act == "gelu_tanh":
        t = torch.tanh(0.7978845608028654 * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * 0.7978845608028654 * (1 + 3 * 0.044715 * z * z)
    s = 1 / (1 + torch.exp(-z))
    return s * (1 + z * (1 - s))


def _plain_linear(s):
    c, w = s["case"], s["w"].float()
    z = s["x"].float() @ (w if c["layout"] == "kn" else w.t())
    if s["bias"] is not None:
        z = z + s["bias"].float()
    y = _act(z, c["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    s["y"].copy_(y)
    if s["z"] is None:
        return [s["y"]]
    s["z"].copy_(z)
    return [s["y"], s["z"]]


def _plain_backward(s):
    c, x, w, dz = s["case"], s["x"].float(), s["w"].float(), s["dz"].float()
    dx = dz @ (w.t() if c["layout"] == "kn" else w)
    if s["zin"] is not None:
        dx = dx * _act_grad(s["zin"].float(), c["act"])
    dw = x.t() @ dz if c["layout"] == "kn" else dz.t() @ x
    db = dz.sum(0)
    if c["accumulate"]:
        dw, db = s["dw"].float() + dw, s["db"].float() + db
    s["dx"].copy_(dx)
    s["dw"].copy_(dw)
    s["db"].copy_(db)
    return [s["dx"], s["dw"], s["db"]]


def _plain_loss(s):
    h, w, adv = s["hyper"], s["weight"], s["adv"]
    it = h["inv_temperature"]
    x = s["logits"].float() * it
    top = x.max(1, keepdim=True).values
    e = torch.exp(x - top)
    total = e.sum(1, keepdim=True)
    live = w != 0
    logp = torch.where(live, (x.gather(1, s["target"][:, None]) - top - torch.log(total))[:, 0], 0.0)
    r = torch.exp(logp - s["old"]) if s["old"] is not None else torch.ones_like(logp)
    clipped = torch.where(adv > 0, r > 1 + h["clip_high"], r < 1 - h["clip_low"]) & (adv != 0)
    loss = -torch.minimum(r * adv, torch.clamp(r, 1 - h["clip_low"], 1 + h["clip_high"]) * adv)
    g = torch.where(clipped, 0.0, -adv * r)
    kl = torch.zeros_like(logp)
    if h["kl_coef"]:
        d = s["ref"] - logp
        kl = torch.expm1(d) - d
        loss = loss + h["kl_coef"] * kl
        g = g - h["kl_coef"] * torch.expm1(d)
    s["logp"].copy_(logp)
    s["stats"].copy_(torch.stack([torch.where(live, w * q, 0.0).sum() for q in (loss, kl, clipped.float(), r)]))
    coef = torch.where(live, w * g, 0.0)[:, None] * (it * h["grad_scale"])
    grad = -coef * (e / total)
    grad.scatter_add_(1, s["target"][:, None], coef)
    s["grad"].copy_(torch.where(live[:, None], grad, 0.0))
    return [s["stats"], s["logp"], s["grad"]]


def _mix(x):
    """The 32-bit integer mixer of the rounding bits, on int64 tensors or ints holding 32-bit values."""
    x = x ^ (x >> 16)
    x = (x * 0x7FEB352D) & MASK32
    x = x ^ (x >> 15)
    x = (x * 0x846CA68B) & MASK32
    return x ^ (x >> 16)


def _bits(n, seed, step, tensor):
    """32 rounding bits for each of a tensor's n elements."""
    key = _mix(_mix(_mix(_mix(tensor) ^ (step & MASK32)) ^ (seed & MASK32)) ^ ((seed >> 32) & MASK32))
    i = torch.arange(n, device="cuda")
    return _mix((i & MASK32) ^ _mix((i >> 32) ^ key))


def _blocks(x):
    n = x.numel()
    pad = -n % STATE_BLOCK
    return torch.cat([x, x.new_zeros(pad)]).view(-1, STATE_BLOCK) if pad else x.view(-1, STATE_BLOCK)


def _to_codes(x, r16):
    """8-bit codes (e4m3) and a power-of-two scale per block of a float tensor.

    r16: 16 random bits per element for stochastic rounding; None rounds to nearest.
    The scale 2^k brings the block's largest magnitude into (224, 448]."""
    n = x.numel()
    b = _blocks(x)
    fine = torch.isfinite(b)
    top = torch.where(fine, b.abs(), 0.0).amax(1)
    e = ((top.view(torch.int32).to(torch.int64) + 0x1FFFFF) >> 23) - 127 - 8
    e = torch.clamp_min(e, -118)
    scale = ((e + 127) << 23).to(torch.int32).view(torch.float32)
    inv = ((127 - e) << 23).to(torch.int32).view(torch.float32)
    y = b * inv[:, None]
    if r16 is not None:
        y = _stochastic(y, _blocks(r16))
    code = torch.where(fine, y, math.nan).to(torch.float8_e4m3fn)
    return code.view(-1)[:n].contiguous(), scale


def _stochastic(y, r16):
    """|y| <= 448 rounded to one of its two e4m3 neighbours, upwards with the probability of the remainder."""
    a = y.abs()
    off = torch.where(a < 0.015625, 0.015625, 0.0)  # below 2^-6 the step stays 2^-9
    t = (a + off).view(torch.int32).to(torch.int64) + (r16 << 4)
    t = (t & 0xFFF00000).to(torch.int32).view(torch.float32)
    return torch.copysign(t - off, y)


def _values(code, scale):
    return (_blocks(code.float()) * scale[:, None]).view(-1)[:code.numel()]


def _adamw_step(t, index, s):
    """One tensor's new (param, m, v, m_scale, v_scale)."""
    c, h, step = s["case"], s["hyper"], s["step"]
    g = t["grad"].float() * s["grad_scale"]
    if c["state"] == 8:
        m, u = _values(t["m"], t["m_scale"]), _values(t["v"], t["v_scale"])
        v = u * u
    else:
        m, v = t["m"], t["v"]
    m = m * h["beta1"] + g * (1 - h["beta1"])
    v = v * h["beta2"] + (g * g) * (1 - h["beta2"])
    u = torch.sqrt(v)
    den = u * (1 / math.sqrt(1 - h["beta2"] ** step)) + h["eps"]
    p = t["param"].float()
    p = p * (1 - h["lr"] * h["weight_decay"]) - (h["lr"] / (1 - h["beta1"] ** step)) * (m / den)
    if c["state"] == 8:
        bits = _bits(p.numel(), s["seed"], step, index)
        m, ms = _to_codes(m, bits & 0xFFFF)
        v, vs = _to_codes(u, bits >> 16)
        return p, m, v, ms, vs
    return p, m, v, None, None


def _plain_adamw(s):
    for i, t in enumerate(s["tensors"]):
        p, m, v, ms, vs = _adamw_step(t, i, s)
        t["param"].copy_(p)
        t["m"].copy_(m)
        t["v"].copy_(v)
        if ms is not None:
            t["m_scale"].copy_(ms)
            t["v_scale"].copy_(vs)
        if "copy" in t:
            t["copy"].copy_(p)
    s["step"] += 1
    return _adamw_outputs(s)


def _adamw_outputs(s):
    """The updated buffers themselves."""
    return {k: f for k, f in s["flat"].items() if k != "grad"}


# --------------------------------------------------------------------------- #
# What a pass cannot do without                                               #
# --------------------------------------------------------------------------- #

def work(case):
    if case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        outs = 1 + (1 if case["z"] else 0) + (1 if case["residual"] else 0)
        return {"bytes": 2 * (M * K + K * N + outs * M * N + (N if case["bias"] else 0)), "flops": 2 * M * N * K}
    if case["op"] == "backward":
        M, N, K = case["M"], case["N"], case["K"]
        ge = (4 if case["grad"] == "f32" else 2) * (2 if case["accumulate"] else 1)
        zin = M * K if case["act"] != "none" else 0
        return {"bytes": 2 * (M * N + M * K + K * N + zin + M * K) + ge * (K * N + N), "flops": 4 * M * N * K + M * N}
    if case["op"] == "loss":
        T, V, es = case["T"], case["V"], 4 if case["dtype"] == "f32" else 2
        live = T * (1 - case["masked"])
        return {"bytes": es * V * (live + T) + T * 32, "flops": 6 * live * V}
    es = {"f32": 4, "bf16": 2, "f16": 2}
    per = 2 * es[case["param"]] + es[case["grad"]] + (16 if case["state"] == 32 else 4 + 16 / STATE_BLOCK)
    per += es[case["copy"]] if case["copy"] else 0
    n = sum(_adamw_sizes(case))
    return {"bytes": per * n, "flops": 15 * n}


# --------------------------------------------------------------------------- #
# The definitions in 64 bits                                                  #
# --------------------------------------------------------------------------- #

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "linear":
        x, w = s["x"].double(), s["w"].double()
        z = torch.matmul(x, w if case["layout"] == "kn" else w.t())
        if s["bias"] is not None:
            z += s["bias"].double()
        y = _exact_act(z, case["act"])
        if s["residual"] is not None:
            y = y + s["residual"].double()
        return [y] if not case["z"] else [y, z]
    if case["op"] == "backward":
        x, w, dz = s["x"].double(), s["w"].double(), s["dz"].double()
        if case["layout"] == "nk":
            w = w.t()
        dx = torch.matmul(dz, w.t())
        if case["act"] != "none":  # the activation's slope, by its own formula
            z = s["zin"].double().requires_grad_(True)
            slope, = torch.autograd.grad(_exact_act(z, case["act"]).sum(), z)
            dx = dx * slope
        dw = torch.matmul(x.t(), dz)
        if case["layout"] == "nk":
            dw = dw.t()
        db = torch.matmul(torch.ones((1, case["M"]), dtype=torch.float64, device="cuda"), dz)[0]
        if case["accumulate"]:
            dw, db = dw + s["dw"].double(), db + s["db"].double()
        return [dx, dw, db]
    if case["op"] == "loss":
        return _exact_loss(s)
    flat = {k: f.double() for k, f in s["flat"].items() if k != "grad"}
    for i, (at, first, n) in enumerate(_places(_adamw_sizes(case))):
        for k, x in _exact_adamw(s, i, s["tensors"][i]).items():
            if k in flat:
                begin = first if k.endswith("_scale") else at
                flat[k][begin:begin + x.numel()] = x
    return flat


def _exact_act(z, act):
    if act == "none":
        return z
    if act == "relu":
        return torch.where(z > 0, z, 0 * z)
    if act == "gelu":
        return z * torch.special.ndtr(z)
    if act == "gelu_tanh":
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    return z * torch.sigmoid(z)


def _exact_loss(s):
    c, h = s["case"], s["hyper"]
    T, V = c["T"], c["V"]
    rows, logp = [], torch.zeros((T,), dtype=torch.float64, device="cuda")
    stats = np.zeros(4)
    step = max(1, (1 << 27) // V)
    for a in range(0, T, step):
        b = min(T, a + step)
        lp = torch.log_softmax(s["logits"][a:b].double() * h["inv_temperature"], 1)
        hot = torch.zeros_like(lp).scatter_(1, s["target"][a:b, None], 1.0)
        mine = (lp * hot).sum(1)
        w, adv = s["weight"][a:b].double(), s["adv"][a:b].double()
        r = torch.exp(mine - (s["old"][a:b].double() if s["old"] is not None else mine))
        lo, hi = 1 - h["clip_low"], 1 + h["clip_high"]
        over = ((adv > 0) & (r > hi)) | ((adv < 0) & (r < lo))
        loss, slope = torch.where(over, -torch.clamp(r, lo, hi) * adv, -r * adv), torch.where(over, 0.0, -r * adv)
        kl = torch.zeros_like(mine)
        if s["ref"] is not None:
            q = torch.exp(s["ref"][a:b].double() - mine)
            kl = q - torch.log(q) - 1
            loss, slope = loss + h["kl_coef"] * kl, slope + h["kl_coef"] * (1 - q)
        on = (w != 0).double()
        logp[a:b] = mine * on
        stats += [float((w * q).sum()) for q in (loss, kl, over.double(), r)]
        grad = (w * slope)[:, None] * (hot - lp.exp()) * (h["inv_temperature"] * h["grad_scale"])
        rows.append(grad.float() if T * V > 1 << 28 else grad)
    return [torch.tensor(stats, device="cuda"), logp, torch.cat(rows)]


def _exact_adamw(s, index, t):
    h, k, n = s["hyper"], s["step"], t["param"].numel()
    eight = s["case"]["state"] == 8

    def stands_for(code, scale):
        return code.double() * scale.double().repeat_interleave(STATE_BLOCK)[:n]

    grad = t["grad"].double() * float(s["grad_scale"])
    m = stands_for(t["m"], t["m_scale"]) if eight else t["m"].double()
    v = stands_for(t["v"], t["v_scale"]).square() if eight else t["v"].double()
    m = torch.lerp(grad, m, h["beta1"])
    v = torch.lerp(grad.square(), v, h["beta2"])
    m_hat, v_hat = m / (1 - h["beta1"] ** k), v / (1 - h["beta2"] ** k)
    p = t["param"].double()
    p = p - h["lr"] * (m_hat / (v_hat.sqrt() + h["eps"]) + h["weight_decay"] * p)
    out = {"param": p, "m": m, "v": v, "copy": p}
    if not eight:
        return out
    # e4m3: steps of 2^-9 below 2^-6 and of an eighth of the power of two above; up where the remainder
    # passes the random fraction that is left over
    bits = _bits(n, s["seed"], k, index)
    for name, x, r in (("m", m, bits % 65536), ("v", v.sqrt(), bits // 65536)):
        whole = torch.zeros((-(-n // STATE_BLOCK) * STATE_BLOCK,), dtype=torch.float64, device="cuda")
        whole[:n] = x.abs()
        frac, power = torch.frexp(whole.view(-1, STATE_BLOCK).max(1).values)   # frac in [0.5, 1)
        scale = torch.ldexp(torch.ones_like(frac), torch.clamp(power - 9 + (frac > 0.875).to(power.dtype), min=-118))
        y = whole[:n] / scale.repeat_interleave(STATE_BLOCK)[:n]
        quantum = torch.ldexp(torch.ones_like(y), torch.clamp(torch.frexp(y).exponent - 4, min=-9))
        # below 2^-6 the 16 random bits stand against the remainder of y + 2^-6, of the same step
        y = torch.floor(y / quantum + r.double() / 65536) * quantum
        out[name], out[name + "_scale"] = torch.where(x < 0, -y, y), scale
    return out
