"""The operators of a residual block's ends and of the vocabulary's loss: cases, plain forms, exact values.

A block's input goes through a root-mean-square norm (with the residual's addition, and an output in 8 bits
for the backward pass), its activations are kept in 8 bits between the passes, and the last hidden states
become a loss over a large vocabulary whose logits are never stored.  Three operators are listed here:
``norm`` (forward and backward), ``checkpoint`` (packing, and a linear layer's gradients from packed
activations) and ``entropy`` (the loss alone, and with its gradients).

With ``own`` false, ``run`` computes them in their plain form: elementary torch operations in float32,
rounded once at the end.  With ``own`` true it calls the library.  ``exact`` gives the same outputs from
the definitions in float64.
"""
from __future__ import annotations

import math

import torch

own = False

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
BLOCK = 128                # elements of a row that share one scale of an 8-bit activation
E4M3 = torch.float8_e4m3fn
EPS = 1e-6


# --------------------------------------------------------------------------- #
# Cases                                                                       #
# --------------------------------------------------------------------------- #

def listed():
    return [
        # one token between two layers while decoding: the residual is added, nothing is kept
        dict(name="norm 1 token", op="norm", M=1, N=8192, dtype="bf16", weight="bf16", residual=True,
             packed=False),
        # a ragged batch of a small model, first norm of the network (no residual), kept for the backward pass
        dict(name="norm 777 odd", op="norm", M=777, N=1523, dtype="f16", weight="f32", residual=False,
             packed=True),
        # a training batch at the largest M_local and K
        dict(name="norm 16384", op="norm", M=16384, N=8192, dtype="bf16", weight="bf16", residual=True,
             packed=True),
        # its gradients: the small model's, gradients in 16 bits
        dict(name="norm backward 777 odd", op="norm_backward", M=777, N=1523, dtype="f16", weight="f32",
             through=False, grad="f16", accumulate=False),
        # the large one's, with the gradient that arrives along the residual, accumulated in f32
        dict(name="norm backward 16384", op="norm_backward", M=16384, N=8192, dtype="bf16", weight="bf16",
             through=True, grad="f32", accumulate=True),
        # a training batch's pre-activations put away in 8 bits
        dict(name="pack 16384 x 3584", op="pack", M=16384, N=3584, dtype="bf16"),
        # gradients of a small layer over a ragged batch from packed pre-activations, 16-bit gradients
        dict(name="packed backward 777 odd", op="packed_backward", M=777, N=1000, K=1523, dtype="bf16",
             layout="kn", act="silu", grad="bf16", accumulate=False),
        # gradients of the benchmark's layer, accumulated in f32 over the data shards
        dict(name="packed backward 4096", op="packed_backward", M=4096, N=3584, K=8192, dtype="bf16",
             layout="nk", act="gelu", grad="f32", accumulate=True),
        # a few generated tokens scored under a small vocabulary
        dict(name="entropy 16 x 8192", op="entropy", T=16, V=8192, K=1024, dtype="bf16", layout="nk",
             masked=0.0, grads=False),
        # a ragged batch of a small model, prompts masked out, weights as the matmul has them (K x V)
        dict(name="entropy 777 x 32768", op="entropy", T=777, V=32768, K=2011, dtype="f16", layout="kn",
             masked=0.3, grads=True),
        # a held-out batch's loss, odd vocabulary
        dict(name="entropy 4096 x 100003 loss", op="entropy", T=4096, V=100003, K=1024, dtype="bf16",
             layout="nk", masked=0.0, grads=False),
        # a training batch with a quarter of it prompt, weight rows gathered
        dict(name="entropy 4096 x 100003", op="entropy", T=4096, V=100003, K=3584, dtype="bf16", layout="nk",
             masked=0.25, grads=True),
    ]


def _log_int(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_backward", "pack", "packed_backward", "entropy", "entropy"])
    dtype = rng.choice(["f16", "bf16"])
    if op == "norm":
        return dict(op=op, M=_log_int(rng, 1, 16384), N=_log_int(rng, 64, 8192), dtype=dtype,
                    weight=rng.choice([dtype, "f32"]), residual=rng.random() < 0.6, packed=rng.random() < 0.6)
    if op == "norm_backward":
        return dict(op=op, M=_log_int(rng, 1, 16384), N=_log_int(rng, 64, 8192), dtype=dtype,
                    weight=rng.choice([dtype, "f32"]), through=rng.random() < 0.6,
                    grad=rng.choice([dtype, "f32"]), accumulate=rng.random() < 0.5)
    if op == "pack":
        return dict(op=op, M=_log_int(rng, 1, 16384), N=_log_int(rng, 64, 8192), dtype=dtype)
    if op == "packed_backward":
        return dict(op=op, M=_log_int(rng, 16, 4096), N=_log_int(rng, 64, 3584), K=_log_int(rng, 64, 8192),
                    dtype=dtype, layout=rng.choice(["kn", "nk"]), act=rng.choice(ACTS),
                    grad=rng.choice([dtype, "f32"]), accumulate=rng.random() < 0.5)
    V, K = _log_int(rng, 64, 100003), _log_int(rng, 64, 3584)
    most = min(4096, int((1 - 0.25) * 4096 * 100003 * 3584 / (V * K)))     # the largest listed case's live tokens
    return dict(op=op, T=_log_int(rng, 1, most), V=V, K=K, dtype=dtype, layout=rng.choice(["kn", "nk"]),
                masked=rng.choice([0.0, 0.3, 0.9]), grads=rng.random() < 0.7)


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


def _room(rows, cols, dtype):
    """An output, pitched like the inputs."""
    return torch.empty((rows, _pitch(cols)), dtype=dtype, device="cuda")[:, :cols]


def _packed_room(M, N):
    """Codes (rows of whole 16 bytes) and scales of an 8-bit activation."""
    codes = torch.zeros((M, (N + 15) // 16 * 16), dtype=E4M3, device="cuda")[:, :N]
    return codes, torch.zeros((M, -(-N // BLOCK)), device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * int(seed) + 29)
    op, dt = case["op"], DT[case["dtype"]]
    s = {"case": case}
    if op in ("norm", "norm_backward"):
        M, N = case["M"], case["N"]
        s["weight"] = (1 + 0.2 * torch.randn((N,), generator=g, device="cuda")).to(DT[case["weight"]])
        s["rstd"] = torch.empty((M,), device="cuda")
    if op == "norm":
        s["x"] = _matrix(M, N, dt, g, 1.5)
        s["r"] = _matrix(M, N, dt, g, 0.5) if case["residual"] else None
        s["h"] = _room(M, N, dt) if case["residual"] else None
        s["y"] = _room(M, N, dt)
        s["codes"], s["scales"] = _packed_room(M, N) if case["packed"] else (None, None)
    elif op == "norm_backward":
        s["h"] = _matrix(M, N, dt, g, 1.5)
        s["rstd"].copy_(torch.rsqrt(s["h"].double().square().mean(1) + EPS))
        s["dy"] = _matrix(M, N, dt, g, 0.1)
        s["dh_in"] = _matrix(M, N, dt, g, 0.1) if case["through"] else None
        s["dh"] = _room(M, N, dt)
        s["dweight"] = torch.randn((N,), generator=g, device="cuda").to(DT[case["grad"]])
    elif op == "pack":
        M, N = case["M"], case["N"]
        # pre-activations: some features are larger than others
        s["x"] = _matrix(M, N, dt, g)
        s["x"].mul_(torch.exp(0.5 * torch.randn((N,), generator=g, device="cuda")).to(dt))
        s["codes"], s["scales"] = _packed_room(M, N)
    elif op == "packed_backward":
        M, N, K = case["M"], case["N"], case["K"]
        s["codes"], s["scales"] = _packed_room(M, K)
        codes, scales = _to_codes(_matrix(M, K, dt, g).float())
        s["codes"].copy_(codes)
        s["scales"].copy_(scales)
        s["w"] = _matrix(*((K, N) if case["layout"] == "kn" else (N, K)), dt, g, K ** -0.5)
        s["dz"] = _matrix(M, N, dt, g, 0.25)
        gdt = DT[case["grad"]]
        s["dx"] = _room(M, K, dt)
        s["dw"] = torch.randn(s["w"].shape, generator=g, device="cuda").to(gdt)
        s["db"] = torch.randn((N,), generator=g, device="cuda").to(gdt)
    else:
        T, V, K = case["T"], case["V"], case["K"]
        s["x"] = _matrix(T, K, dt, g)
        s["w"] = _matrix(*((K, V) if case["layout"] == "kn" else (V, K)), dt, g, 2.5 * K ** -0.5)
        s["target"] = torch.randint(0, V, (T,), generator=g, device="cuda")
        keep = torch.rand((T,), generator=g, device="cuda") >= case["masked"]
        s["weight"] = keep.float() / max(1.0, float(keep.sum()))
        s["grad_scale"] = 1024.0 if case["dtype"] == "f16" else 1.0
        s["stats"] = torch.empty((2,), device="cuda")
        s["loss"], s["lse"] = (torch.empty((T,), device="cuda") for _ in range(2))
        s["dx"] = _room(T, K, dt) if case["grads"] else None
        s["dw"] = _room(*s["w"].shape, dt) if case["grads"] else None
    return s


# --------------------------------------------------------------------------- #
# One pass                                                                    #
# --------------------------------------------------------------------------- #

def run(state):
    op = state["case"]["op"]
    return globals()[("_own_" if own else "_plain_") + op](state)


def _ld(x):
    return x.stride(0) if x is not None else 0


def _bytes(s, n):
    """Device scratch of a call, allocated once by a program and kept for its later calls."""
    if "workspace" not in s:
        s["workspace"] = torch.empty((n,), dtype=torch.uint8, device="cuda")
    return s["workspace"]


def _own_norm(s):
    import gemm_gather_gb300 as gg
    c = s["case"]
    gg.rms_norm(s["x"], _ld(s["x"]), s["r"], _ld(s["r"]), s["weight"], EPS, s["h"], _ld(s["h"]), s["y"], _ld(s["y"]),
                s["codes"], _ld(s["codes"]), s["scales"], _ld(s["scales"]), s["rstd"], c["M"], c["N"], s["x"].dtype)
    return _norm_outputs(s)


def _own_norm_backward(s):
    import gemm_gather_gb300 as gg
    c = s["case"]
    work = _bytes(s, gg.rms_norm_backward_workspace(c["M"], c["N"]))
    gg.rms_norm_backward(s["dy"], _ld(s["dy"]), s["h"], _ld(s["h"]), s["rstd"], s["weight"], s["dh_in"], _ld(s["dh_in"]),
                         s["dh"], _ld(s["dh"]), s["dweight"], s["dweight"].dtype, c["accumulate"], work,
                         c["M"], c["N"], s["dy"].dtype)
    return [s["dh"], s["dweight"]]


def _own_pack(s):
    import gemm_gather_gb300 as gg
    c = s["case"]
    gg.pack8(s["x"], _ld(s["x"]), s["codes"], _ld(s["codes"]), s["scales"], _ld(s["scales"]), c["M"], c["N"], s["x"].dtype)
    return [s["codes"], s["scales"]]


def _own_packed_backward(s):
    import gemm_gather_gb300 as gg
    c = s["case"]
    work = _bytes(s, gg.linear_backward8_workspace(c["M"], c["K"]))
    gg.linear_backward8(s["dz"], _ld(s["dz"]), s["codes"], _ld(s["codes"]), s["scales"], _ld(s["scales"]), c["act"],
                        s["w"], _ld(s["w"]), c["layout"], s["dx"], _ld(s["dx"]), s["dw"], _ld(s["dw"]), s["db"],
                        s["dw"].dtype, c["accumulate"], work, c["M"], c["N"], c["K"], s["dz"].dtype)
    return [s["dx"], s["dw"], s["db"]]


def _own_entropy(s):
    import gemm_gather_gb300 as gg
    c = s["case"]
    work = _bytes(s, gg.linear_cross_entropy_workspace(c["T"], c["V"], c["K"], gradients=c["grads"]))
    gg.linear_cross_entropy(s["x"], _ld(s["x"]), s["w"], _ld(s["w"]), c["layout"], s["target"], s["weight"],
                            s["stats"], s["loss"], s["lse"], s["dx"], _ld(s["dx"]), s["dw"], _ld(s["dw"]), s["x"].dtype,
                            False, work, c["T"], c["V"], c["K"], s["x"].dtype, grad_scale=s["grad_scale"])
    return _entropy_outputs(s)


def _norm_outputs(s):
    out = [s["y"], s["rstd"]]
    if s["h"] is not None:
        out.append(s["h"])
    if s["codes"] is not None:
        out += [s["codes"], s["scales"]]
    return out


def _entropy_outputs(s):
    out = [s["stats"], s["loss"], s["lse"]]
    return out + [s["dx"], s["dw"]] if s["case"]["grads"] else out


def _blocks(x):
    pad = -x.shape[1] % BLOCK
    if pad:
        x = torch.cat([x, x.new_zeros((x.shape[0], pad))], 1)
    return x.view(x.shape[0], -1, BLOCK)


def _to_codes(x):
    """Codes (e4m3, to nearest) of a float32 matrix and a power-of-two scale for each BLOCK elements of a
    row: the one that brings the block's largest magnitude into (224, 448]."""
    b = _blocks(x)
    fine = torch.isfinite(b)
    top = torch.where(fine, b.abs(), 0.0).amax(2)
    e = ((top.view(torch.int32).to(torch.int64) + 0x1FFFFF) >> 23) - 127 - 8
    e = torch.clamp_min(e, -118)
    scale = ((e + 127) << 23).to(torch.int32).view(torch.float32)
    inv = ((127 - e) << 23).to(torch.int32).view(torch.float32)
    code = torch.where(fine, b * inv[:, :, None], math.nan).to(E4M3)
    return code.view(x.shape[0], -1)[:, :x.shape[1]], scale


def _values(codes, scales):
    return (_blocks(codes.float()) * scales[:, :, None]).view(codes.shape[0], -1)[:, :codes.shape[1]]


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


def _plain_norm(s):
    x = s["x"].float()
    if s["r"] is not None:
        s["h"].copy_(x + s["r"].float())
        x = s["h"].float()
    rstd = 1 / torch.sqrt((x * x).mean(1) + EPS)
    s["rstd"].copy_(rstd)
    s["y"].copy_(x * rstd[:, None] * s["weight"].float())
    if s["codes"] is not None:  # what the next layer reads, in 8 bits
        codes, scales = _to_codes(s["y"].float())
        s["codes"].copy_(codes)
        s["scales"].copy_(scales)
    return _norm_outputs(s)


def _plain_norm_backward(s):
    h, dy, rstd = s["h"].float(), s["dy"].float(), s["rstd"][:, None]
    u = h * rstd
    gy = dy * s["weight"].float()
    dh = rstd * (gy - u * (gy * u).mean(1, keepdim=True))
    if s["dh_in"] is not None:
        dh = dh + s["dh_in"].float()
    s["dh"].copy_(dh)
    dweight = (dy * u).sum(0)
    if s["case"]["accumulate"]:
        dweight = dweight + s["dweight"].float()
    s["dweight"].copy_(dweight)
    return [s["dh"], s["dweight"]]


def _plain_pack(s):
    codes, scales = _to_codes(s["x"].float())
    s["codes"].copy_(codes)
    s["scales"].copy_(scales)
    return [s["codes"], s["scales"]]


def _plain_packed_backward(s):
    c, p, w, dz = s["case"], _values(s["codes"], s["scales"]), s["w"].float(), s["dz"].float()
    x = _act(p, c["act"])
    dx = dz @ (w.t() if c["layout"] == "kn" else w)
    if c["act"] != "none":
        dx = dx * _act_grad(p, c["act"])
    dw = x.t() @ dz if c["layout"] == "kn" else dz.t() @ x
    db = dz.sum(0)
    if c["accumulate"]:
        dw, db = s["dw"].float() + dw, s["db"].float() + db
    s["dx"].copy_(dx)
    s["dw"].copy_(dw)
    s["db"].copy_(db)
    return [s["dx"], s["dw"], s["db"]]


def _plain_entropy(s):
    c, x, w, t, tw = s["case"], s["x"].float(), s["w"].float(), s["target"], s["weight"]
    if c["layout"] == "nk":
        w = w.t()
    live = tw != 0
    z = x @ w
    top = z.max(1, keepdim=True).values
    mine = z.gather(1, t[:, None])[:, 0]
    z.sub_(top).exp_()
    total = z.sum(1, keepdim=True)
    lse = (top + torch.log(total))[:, 0]
    loss = torch.where(live, lse - mine, 0.0)
    s["loss"].copy_(loss)
    s["lse"].copy_(torch.where(live, lse, 0.0))
    s["stats"].copy_(torch.stack([(loss.double() * tw.double()).sum(), tw.double().sum()]))
    if not c["grads"]:
        return _entropy_outputs(s)
    coef = torch.where(live, tw, 0.0)[:, None] * s["grad_scale"]
    z.mul_(coef / total)
    z.scatter_add_(1, t[:, None], -coef)
    s["dx"].copy_(z @ w.t())
    s["dw"].copy_(x.t() @ z if c["layout"] == "kn" else z.t() @ x)
    return _entropy_outputs(s)


# --------------------------------------------------------------------------- #
# What a pass cannot do without                                               #
# --------------------------------------------------------------------------- #

def work(case):
    op, es = case["op"], {"f32": 4, "bf16": 2, "f16": 2}
    if op == "norm":
        M, N = case["M"], case["N"]
        per = 4 + (4 if case["residual"] else 0) + (1 + 4 / BLOCK if case["packed"] else 0)
        return {"bytes": per * M * N + 4 * M + es[case["weight"]] * N, "flops": 5 * M * N}
    if op == "norm_backward":
        M, N = case["M"], case["N"]
        grads = es[case["grad"]] * (2 if case["accumulate"] else 1)
        return {"bytes": (8 if case["through"] else 6) * M * N + 4 * M + (es[case["weight"]] + grads) * N,
                "flops": 9 * M * N}
    if op == "pack":
        return {"bytes": (3 + 4 / BLOCK) * case["M"] * case["N"], "flops": 2 * case["M"] * case["N"]}
    if op == "packed_backward":
        M, N, K = case["M"], case["N"], case["K"]
        ge = es[case["grad"]] * (2 if case["accumulate"] else 1)
        return {"bytes": 2 * (M * N + K * N + M * K) + (1 + 4 / BLOCK) * M * K + ge * (K * N + N),
                "flops": 4 * M * N * K + M * N}
    T, V, K = case["T"], case["V"], case["K"]
    live = T * (1 - case["masked"])
    if not case["grads"]:
        return {"bytes": 2 * (live * K + V * K) + 20 * T, "flops": 2 * live * V * K}
    # logits once, and the two products of their gradient
    return {"bytes": 2 * (live * K + V * K + T * K + V * K) + 20 * T, "flops": 6 * live * V * K}


# --------------------------------------------------------------------------- #
# The definitions in 64 bits                                                  #
# --------------------------------------------------------------------------- #

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        return _exact_norm(s)
    if op == "norm_backward":
        # the gradient of <y(h), dy> by differentiating the norm itself, in 64 bits
        h, w = s["h"].double().requires_grad_(True), s["weight"].double().requires_grad_(True)
        y = h / torch.sqrt(h.pow(2).sum(1, keepdim=True) / case["N"] + EPS) * w
        dh, dw = torch.autograd.grad(y, (h, w), s["dy"].double())
        if s["dh_in"] is not None:
            dh = dh + s["dh_in"].double()
        return [dh, dw + s["dweight"].double() if case["accumulate"] else dw]
    if op == "pack":
        return list(_exact_codes(s["x"]))
    if op == "packed_backward":
        scale = s["scales"].double().repeat_interleave(BLOCK, 1)[:, :case["K"]]
        p = (s["codes"].double() * scale).requires_grad_(True)
        x = _exact_act(p, case["act"])
        w, dz = s["w"].double(), s["dz"].double()
        if case["layout"] == "nk":
            w = w.t()
        dx, = torch.autograd.grad(x, p, torch.matmul(dz, w.t()))
        dw = torch.matmul(x.detach().t(), dz)
        if case["layout"] == "nk":
            dw = dw.t()
        db = torch.matmul(torch.ones((1, case["M"]), dtype=torch.float64, device="cuda"), dz)[0]
        if case["accumulate"]:
            dw, db = dw + s["dw"].double(), db + s["db"].double()
        return [dx, dw, db]
    return _exact_entropy(s)


def _exact_act(z, act):
    if act == "none":
        return z * 1.0
    if act == "relu":
        return torch.where(z > 0, z, 0 * z)
    if act == "gelu":
        return z * torch.special.ndtr(z)
    if act == "gelu_tanh":
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    return z * torch.sigmoid(z)


def _power_of_two(e):
    """2^e in float64, by its bits (a power function may be a step off)."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_codes(x):
    """e4m3 by its steps: 2^-9 below 2^-6, an eighth of the power of two above; ties to even."""
    M, N = x.shape
    whole = torch.zeros((M, -(-N // BLOCK) * BLOCK), dtype=torch.float64, device="cuda")
    whole[:, :N] = x.double()
    frac, power = torch.frexp(whole.abs().view(M, -1, BLOCK).max(2).values)   # frac in [0.5, 1)
    power = torch.where(frac == 0, -200, power)     # nothing but zeros: the least scale
    scale = _power_of_two(torch.clamp(power - 9 + (frac > 0.875).to(power.dtype), min=-118))
    y = whole[:, :N] / scale.repeat_interleave(BLOCK, 1)[:, :N]
    quantum = _power_of_two(torch.clamp(torch.frexp(y).exponent - 4, min=-9))
    return torch.round(y / quantum) * quantum, scale


def _exact_norm(s):
    c = s["case"]
    h = s["x"].double()
    total = h
    if s["r"] is not None:
        total = h + s["r"].double()
        h = total.to(s["x"].dtype).double()     # the sum is kept in 16 bits, and the norm is of what is kept
    r = torch.rsqrt(torch.linalg.vecdot(h, h) / c["N"] + EPS)
    y = torch.einsum("mn,m,n->mn", h, r, s["weight"].double())
    out = [y, r]
    if s["r"] is not None:
        out.append(total)
    if c["packed"]:
        out += list(_exact_codes(y.to(s["x"].dtype)))
    return out


def _exact_entropy(s):
    c = s["case"]
    T, V = c["T"], c["V"]
    on = (s["weight"] != 0)
    x, w, tw = s["x"].double(), s["w"].double(), s["weight"].double()
    dx, dw = (torch.zeros(t.shape, dtype=torch.float64, device="cuda") for t in (x, w))
    loss, lse = (torch.zeros((T,), dtype=torch.float64, device="cuda") for _ in range(2))
    step = max(1, (1 << 28) // V)
    for a in range(0, T, step):
        xs = x[a:a + step]
        z = torch.matmul(xs, w if c["layout"] == "kn" else w.t())
        top = torch.logsumexp(z, 1)
        lse[a:a + step] = top
        z -= top[:, None]
        loss[a:a + step] = -torch.take_along_dim(z, s["target"][a:a + step, None], 1)[:, 0]
        if c["grads"]:
            z = z.exp_()
            z[torch.arange(xs.shape[0], device="cuda"), s["target"][a:a + step]] -= 1.0
            z *= (tw[a:a + step] * s["grad_scale"])[:, None]
            dx[a:a + step] = torch.matmul(z, w.t() if c["layout"] == "kn" else w)
            dw += torch.matmul(xs.t(), z) if c["layout"] == "kn" else torch.matmul(z.t(), xs)
    loss, lse = loss * on, lse * on
    out = [torch.stack([torch.dot(loss, tw), tw.sum()]), loss, lse]
    return out + [dx, dw] if c["grads"] else out
