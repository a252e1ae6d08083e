"""Cases of the operators that train and serve a mixture-of-experts block, with their plain forms.

* ``join``   -- the residual stream between two blocks: the norm behind a block, its gate and scale, the
                residual addition and the next block's norm, forward and backward.
* ``adamw``  -- one AdamW step over all tensors of a block (or of many), with the gradients' global norm,
                states in 32 bits or in 8 (blocks of 32: E4M3 elements, one power-of-two scale).
* ``w4``     -- few tokens through SwiGLU experts whose weights are 4-bit integers with a scale and a zero
                point for each group of 32, 64 or 128 along the contraction; ``matvec`` is one such product.

``run`` computes them in their plain form (elementary torch operations in 32 bits, rounded once)
unless ``own`` is true, when it makes the library's calls.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
EPS = 1e-5
NORMS = {"none": 0, "layer": 1, "rms": 2}
RES, BRANCH = 0.9, 0.7               # residual and branch scale
LR, B1, B2, ADAM_EPS, DECAY = 1e-3, 0.9, 0.95, 1e-8, 0.1
DONE, SEED = 100, 12345              # steps before this one; seed of the stochastic rounding
BLOCK = 32                           # elements of an 8-bit state's scale
LARGEST_JOIN = 16384 * 2048
LARGEST_ADAM = 64 * 3 * 2048 * 512   # parameters of the largest step
LARGEST_W4 = 256 * 3 * 2048 * 512    # weights of the largest expert layer


def listed():
    return [
        # between two blocks of a decode step, 16 sequences: latency
        dict(name="join decode", op="join", T=16, d=2048, stream="bf16", branch="bf16", post="rms", pre="rms", gate=False,
             bias=False, backward=False),
        # one training step of the large workload, forward
        dict(name="join forward large", op="join", T=16384, d=2048, stream="bf16", branch="bf16", post="rms", pre="rms",
             gate=True, bias=False, backward=False),
        # ... and backward, with layer norms and every gradient that there is
        dict(name="join backward large", op="join", T=16384, d=2048, stream="bf16", branch="bf16", post="layer", pre="layer",
             gate=True, bias=True, backward=True),
        # residual stream in fp32, rows and width that fill no tile (the skew workload's sizes)
        dict(name="join backward fp32 stream", op="join", T=20000, d=1000, stream="fp32", branch="bf16", post="rms", pre="layer",
             gate=True, bias=True, backward=True),
        # one block of the toy workload, gradients clipped: latency
        dict(name="adamw toy", op="adamw", E=4, d=64, h=128, blocks=1, experts=True, bits=32, p="fp32", g="fp32", clip=True),
        # norms and routers of 24 fine-grained blocks: 72 tensors, most of them small
        dict(name="adamw norms and routers", op="adamw", E=128, d=2048, h=768, blocks=24, experts=False, bits=32, p="copy",
             g="fp32", clip=False),
        # one block of the medium workload, fp32 master weights with their bf16 copy, gradients clipped
        dict(name="adamw medium", op="adamw", E=64, d=2048, h=512, blocks=1, experts=True, bits=32, p="copy", g="fp32",
             clip=True),
        # one block of the skew workload with 8-bit states and bf16 weights
        dict(name="adamw skew 8 bits", op="adamw", E=64, d=1000, h=1000, blocks=1, experts=True, bits=8, p="bf16", g="fp32",
             clip=False),
        # one projection of one token (the projection study's 4096 x 4096)
        dict(name="w4 matvec", op="matvec", T=1, N=4096, K=4096, group=128),
        # one token through the fine-grained layer
        dict(name="w4 one token", op="w4", T=1, E=128, k=8, d=2048, h=768, group=128),
        # one decode step of 16 sequences
        dict(name="w4 decode", op="w4", T=16, E=128, k=8, d=2048, h=768, group=32),
        # one decode step of 64 sequences at the large workload's sizes
        dict(name="w4 decode large", op="w4", T=64, E=256, k=8, d=2048, h=512, group=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["join", "adamw", "w4", "matvec"])
    if op == "join":
        d = _log(rng, 64, 8192)
        if rng.random() < 0.5:
            d = max(64, d // 64 * 64)
        stream, branch = rng.choice([("bf16", "bf16"), ("fp32", "bf16"), ("fp32", "fp32")])
        post = rng.choice(["none", "layer", "rms"])
        return dict(op=op, T=_log(rng, 1, min(32768, LARGEST_JOIN // (2 * d))), d=d, stream=stream, branch=branch, post=post,
                    pre=rng.choice(["layer", "rms", "none"] if post != "none" else ["layer", "rms"]), gate=rng.random() < 0.5,
                    bias=rng.random() < 0.5, backward=rng.random() < 0.6)
    if op == "adamw":
        E, d, h = _log(rng, 2, 64), _log(rng, 33, 2048), _log(rng, 32, 1024)
        while E * 3 * d * h > LARGEST_ADAM // 2:
            E = max(1, E // 2)
        blocks = rng.randint(1, 4)
        while blocks > 1 and blocks * E * 3 * d * h > LARGEST_ADAM // 2:
            blocks -= 1
        return dict(op=op, E=E, d=d, h=h, blocks=blocks, experts=rng.random() < 0.8, bits=rng.choice([32, 8]),
                    p=rng.choice(["fp32", "copy", "bf16"]), g=rng.choice(["fp32", "bf16"]), clip=rng.random() < 0.5)
    group = rng.choice([32, 64, 128])
    if op == "matvec":
        return dict(op=op, T=_log(rng, 1, 32), N=_log(rng, 64, 8192), K=_log(rng, 64, 8192), group=group)
    E = _log(rng, 4, 256)
    k = rng.randint(1, min(8, E))
    d, h = _log(rng, 64, 4096), _log(rng, 64, 2048)
    if rng.random() < 0.5:
        d, h = max(64, d // 64 * 64), max(64, h // 64 * 64)
    while E > k and E * 3 * d * h > LARGEST_W4 // 2:
        E = max(k, E // 2)
    return dict(op=op, T=_log(rng, 1, 64), E=E, k=k, d=d, h=h, group=group)


# ------------------------------------------------------------------------------------- inputs
_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _normal(g, *shape, dtype=torch.float32, std=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * std).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = dict(case)
    {"join": _prepare_join, "adamw": _prepare_adamw, "w4": _prepare_w4, "matvec": _prepare_matvec}[case["op"]](s, g)
    return s


def _prepare_join(s, g):
    T, d, tx, ty = s["T"], s["d"], _TYPES[s["stream"]], _TYPES[s["branch"]]
    weight = lambda on, mean, std: mean + std * _normal(g, d) if on else None  # noqa: E731
    s["post_gamma"] = weight(s["post"] != "none", 1.0, 0.2)
    s["post_beta"] = weight(s["post"] == "layer" and s["bias"], 0.0, 0.1)
    s["gate_w"] = weight(s["gate"], 0.3, 0.2)
    s["pre_gamma"] = weight(s["pre"] != "none", 1.0, 0.2)
    s["pre_beta"] = weight(s["pre"] == "layer" and s["bias"], 0.0, 0.1)
    spread = torch.exp(0.3 * _normal(g, d))
    s["y"] = (0.5 * _normal(g, T, d) * spread + 0.1 * _normal(g, d)).to(ty)
    stream = (_normal(g, T, d) * spread + 0.3 * _normal(g, d)).to(tx)
    if not s["backward"]:
        s["x"] = stream
    else:
        # what the forward left: the joined rows and the statistics of both norms
        s["r"] = stream
        stats = []
        for kind, t in ((s["post"], s["y"]), (s["pre"], s["r"])):
            t = t.double()
            mean = t.mean(1) if kind == "layer" else torch.zeros(T, dtype=torch.float64, device=DEV)
            var = (t - mean[:, None]).square().mean(1)
            stats += [mean, torch.ones_like(var) if kind == "none" else 1.0 / torch.sqrt(var + EPS)]
        s["stats"] = torch.stack(stats).float()
        s["dr"] = _normal(g, T, d, dtype=tx)
        s["dn"] = _normal(g, T, d, dtype=ty) if s["pre"] != "none" else None
    if own:
        from ragged_grouped_gemm_device_gb300 import _lib as L
        new = lambda *shape, dtype=torch.float32: torch.empty(*shape, dtype=dtype, device=DEV)  # noqa: E731
        if not s["backward"]:
            s["out_r"] = new(T, d, dtype=tx)
            s["out_n"] = new(T, d, dtype=ty) if s["pre"] != "none" else None
        else:
            s["dx"], s["dy"] = new(T, d, dtype=tx), new(T, d, dtype=ty)
            for name in ("post_gamma", "post_beta", "gate_w", "pre_gamma", "pre_beta"):
                s["d_" + name] = None if s[name] is None else new(d)
            s["ws"] = new(max(1, L.moe_workspace_bytes(L.OP_RESIDUAL_NORM_BWD, T, 1, 1, d)), dtype=torch.uint8)


def _sizes(case):
    """Elements of each tensor of the step: those with weight decay first (router, up and gate, down), then the norms'."""
    E, d, h = case["E"], case["d"], case["h"]
    matrices = [E * d] + ([E * 2 * h * d, E * h * d] if case["experts"] else [])
    return matrices * case["blocks"], [d, d] * case["blocks"]


def _up32(n):
    return (n + BLOCK - 1) // BLOCK * BLOCK


def _prepare_adamw(s, g):
    decayed, plain = _sizes(s)
    s["sizes"] = decayed + plain
    starts = [0]
    for n in s["sizes"]:
        starts.append(starts[-1] + _up32(n))
    s["starts"], total = starts[:-1], starts[-1]
    s["split"] = starts[len(decayed)]
    live = torch.zeros(total, dtype=torch.bool, device=DEV)   # the rest is room between two tensors
    for at, n in zip(s["starts"], s["sizes"]):
        live[at:at + n] = True
    # the spread of gradients differs from row to row of a weight
    size = torch.exp(_normal(g, total // BLOCK)).repeat_interleave(BLOCK) * 1e-3
    s["g"] = (torch.where(live, _normal(g, total) * size, 0.0)).to(_TYPES[s["g"]])
    p = torch.where(live, _normal(g, total, std=0.02), 0.0)
    s["p_flat"] = p.to(torch.bfloat16) if s["p"] == "bf16" else p
    s["copy"] = p.to(torch.bfloat16) if s["p"] == "copy" else None
    m = torch.where(live, 0.3 * _normal(g, total) * size, 0.0)
    v = torch.where(live, size * size * (0.3 + torch.rand(total, generator=g, device=DEV)), 0.0)
    del p, size
    s["steps"] = DONE
    s["max_norm"] = 0.5e-3 * math.sqrt(sum(s["sizes"])) if s["clip"] else None
    if s["bits"] == 8:
        s["m"], s["m_scale"] = _store8(m, torch.full((total,), 0.5, device=DEV), False)
        s["v"], s["v_scale"] = _store8(torch.sqrt(v), torch.full((total,), 0.5, device=DEV), True)
    else:
        s["m"], s["v"] = m, v
    if own:
        from ragged_grouped_gemm_device_gb300.optim import AdamW
        part = lambda t: [t[a:a + n] for a, n in zip(s["starts"], s["sizes"])]  # noqa: E731
        s["grads"] = part(s["g"])
        s["opt"] = o = AdamW(part(s["p_flat"]), lr=LR, betas=(B1, B2), eps=ADAM_EPS,
                             weight_decay=[DECAY] * len(decayed) + [0.0] * len(plain), state_bits=s["bits"],
                             copies=None if s["copy"] is None else part(s["copy"]), max_norm=s["max_norm"], seed=SEED)
        # a run that goes on from a checkpoint
        o.steps = DONE
        o.m.copy_(s["m"].view(o.m.dtype))
        o.v.copy_(s["v"].view(o.v.dtype))
        if s["bits"] == 8:
            o.m_scale.copy_(s["m_scale"].view(o.m_scale.dtype))
            o.v_scale.copy_(s["v_scale"].view(o.v_scale.dtype))


def _quantized(s, g, name, matrices, N, K):
    """A 4-bit checkpoint's tensors of [matrices, N, K] weights of spread K^-1/2: codes two to a byte (the even element
    low), a scale and a zero point for each group of a row."""
    group = s["group"]
    groups = (K + group - 1) // group
    c = torch.empty(matrices, N, (K + 1) // 2, dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 26) // (N * K))
    for e in range(0, matrices, step):
        n = min(step, matrices - e)
        q = torch.clamp(torch.round(torch.randn(n, N, 2 * ((K + 1) // 2), generator=g, device=DEV) * 2.7 + 7.5), 0, 15).to(torch.uint8)
        c[e:e + n] = q[..., 0::2] | (q[..., 1::2] << 4)
    s[name] = c
    s[name + "_scale"] = ((0.8 + 0.4 * torch.rand(matrices, N, groups, generator=g, device=DEV)) * (K ** -0.5 / 2.7)).to(torch.bfloat16)
    s[name + "_zero"] = torch.randint(6, 10, (matrices, N, groups), generator=g, device=DEV, dtype=torch.uint8)


def _prepare_w4(s, g):
    T, E, k, d, h = (s[n] for n in ("T", "E", "k", "d", "h"))
    s["x"] = (_normal(g, T, d) * torch.exp(0.5 * _normal(g, d))).to(torch.bfloat16)
    _quantized(s, g, "ug", 2 * E, h, d)      # matrices 2e: gate of expert e, 2e + 1: up
    _quantized(s, g, "down", E, d, h)
    top = torch.sort(_normal(g, T, E) + 0.5 * _normal(g, E), dim=1, descending=True, stable=True)
    s["ids"] = top.indices[:, :k].to(torch.int32).contiguous()
    s["weights"] = torch.softmax(top.values[:, :k], dim=1).contiguous()
    if own:
        from ragged_grouped_gemm_device_gb300 import _lib as L
        s["w_ug"], s["w_down"] = _packed(s, "ug", 2 * E, h, d), _packed(s, "down", E, d, h)
        s["out"] = torch.empty(T, d, dtype=torch.bfloat16, device=DEV)
        s["ws"] = torch.empty(max(1, L.moe_workspace_bytes(L.OP_W4_DECODE, T, k, E, d, h)), dtype=torch.uint8, device=DEV)


def _packed(s, name, matrices, N, K):
    from ragged_grouped_gemm_device_gb300 import _lib as L
    w = torch.empty(L.moe_workspace_bytes(L.OP_W4_WEIGHTS, 0, 1, matrices, K, N, s["group"]), dtype=torch.uint8, device=DEV)
    L.moe_w4_pack(s[name], s[name + "_scale"], s[name + "_zero"], matrices, N, K, s["group"], w)
    return w


def _prepare_matvec(s, g):
    T, N, K = s["T"], s["N"], s["K"]
    s["x"] = _normal(g, T, K, dtype=torch.bfloat16)
    _quantized(s, g, "w", 1, N, K)
    if own:
        s["packed"] = _packed(s, "w", 1, N, K)
        s["out"] = torch.empty(T, N, dtype=torch.bfloat16, device=DEV)


# ------------------------------------------------------------------------------- the operators
def run(s):
    return (_own if own else _plain)[s["op"]](s)


def _own_join(s):
    from ragged_grouped_gemm_device_gb300 import _lib as L
    T, d, post, pre = s["T"], s["d"], NORMS[s["post"]], NORMS[s["pre"]]
    if not s["backward"]:
        L.moe_residual_norm_fwd(s["x"], s["y"], post, s["post_gamma"], s["post_beta"], s["gate_w"], pre, s["pre_gamma"],
                                s["pre_beta"], T, d, EPS, RES, BRANCH, s["out_r"], s["out_n"])
        return {"r": s["out_r"], "n": s["out_n"]}
    L.moe_residual_norm_bwd(s["dn"], s["dr"], s["r"], s["y"], post, s["post_gamma"], s["post_beta"], s["gate_w"], pre,
                            s["pre_gamma"], s["stats"], T, d, RES, BRANCH, s["dx"], s["dy"], s["d_post_gamma"],
                            s["d_post_beta"], s["d_gate_w"], s["d_pre_gamma"], s["d_pre_beta"], s["ws"])
    return {n: s[n] for n in ("dx", "dy", "d_post_gamma", "d_post_beta", "d_gate_w", "d_pre_gamma", "d_pre_beta")}


def _own_adamw(s):
    o = s["opt"]
    norm = o.step(s["grads"])
    out = {"p": s["p_flat"], "copy": s["copy"], "norm": norm}
    if s["bits"] == 32:
        return {**out, "m": o.m, "v": o.v}
    return {**out, **_values8(o.m, o.m_scale, o.v, o.v_scale)}


def _own_w4(s):
    from ragged_grouped_gemm_device_gb300 import _lib as L
    L.moe_w4_swiglu_decode(s["x"], s["ids"], s["weights"], s["T"], s["k"], s["E"], s["d"], s["h"], s["group"], s["w_ug"],
                           s["w_down"], s["out"], s["ws"])
    return s["out"]


def _own_matvec(s):
    from ragged_grouped_gemm_device_gb300 import _lib as L
    L.moe_w4_matvec(s["x"], None, s["T"], 1, 1, s["N"], s["K"], s["group"], s["packed"], s["out"])
    return s["out"]


_own = {"join": _own_join, "adamw": _own_adamw, "w4": _own_w4, "matvec": _own_matvec}


def _norm(kind, t):
    """fp32 rows normalised."""
    c = t - t.mean(1, keepdim=True) if kind == "layer" else t
    return c * torch.rsqrt((c * c).mean(1, keepdim=True) + EPS)


def _affine(t, gamma, beta):
    t = t if gamma is None else t * gamma
    return t if beta is None else t + beta


def _plain_join(s):
    gate = BRANCH if s["gate_w"] is None else BRANCH * s["gate_w"]
    ty = s["y"].dtype
    y = s["y"].float()
    if not s["backward"]:
        z = _affine(y if s["post"] == "none" else _norm(s["post"], y), s["post_gamma"], s["post_beta"])
        r = (RES * s["x"].float() + gate * z).to(s["x"].dtype)
        if s["pre"] == "none":
            return {"r": r, "n": None}
        return {"r": r, "n": _affine(_norm(s["pre"], r.float()), s["pre_gamma"], s["pre_beta"]).to(ty)}
    mean1, rstd1, mean2, rstd2 = (t[:, None] for t in s["stats"])
    D = s["dr"].float()
    out = dict.fromkeys(("dx", "dy", "d_post_gamma", "d_post_beta", "d_gate_w", "d_pre_gamma", "d_pre_beta"))
    if s["pre"] != "none":
        dn, rhat = s["dn"].float(), (s["r"].float() - mean2) * rstd2
        D = D + _norm_back(s["pre"], dn * s["pre_gamma"], rhat, rstd2)
        out["d_pre_gamma"] = (dn * rhat).sum(0)
        out["d_pre_beta"] = None if s["pre_beta"] is None else dn.sum(0)
    yhat = (y - mean1) * rstd1
    dz = gate * D
    out["dx"] = (RES * D).to(s["r"].dtype)
    if s["gate_w"] is not None:
        out["d_gate_w"] = (BRANCH * D * _affine(yhat, s["post_gamma"], s["post_beta"])).sum(0)
    if s["post"] == "none":
        out["dy"] = dz.to(ty)
        return out
    out["d_post_gamma"] = (dz * yhat).sum(0)
    out["d_post_beta"] = None if s["post_beta"] is None else dz.sum(0)
    out["dy"] = _norm_back(s["post"], dz * s["post_gamma"], yhat, rstd1).to(ty)
    return out


def _norm_back(kind, d, hat, rstd):
    d = d - hat * (d * hat).mean(1, keepdim=True) - (d.mean(1, keepdim=True) if kind == "layer" else 0.0)
    return rstd * d


def _mix(x):
    """A 32-bit mixing function (the finalizer of MurmurHash3) of int64 values."""
    m = 0xFFFFFFFF
    x = x & m
    x = ((x ^ (x >> 16)) * 0x85EBCA6B) & m
    x = ((x ^ (x >> 13)) * 0xC2B2AE35) & m
    return x ^ (x >> 16)


def _random(s):
    """The 32 bits that decide the rounding of each element: a hash of the seed, the step, the tensor and the element's
    place in it. Low half: m, high half: v, the middle 16 bits: bf16 weights."""
    key = [_mix(SEED ^ _mix(0x9E3779B9 * s["steps"] + t)) for t in range(len(s["sizes"]))]
    i = torch.arange(_up32(max(s["sizes"])), device=DEV) * 0x9E3779B9
    return torch.cat([_mix(i[:_up32(n)] + k) for n, k in zip(s["sizes"], key)])


def _power(e):
    """2^e as fp32 for int32 e from -127 to 127."""
    return torch.where(e > -127, ((e + 127) << 23), 1 << 22).view(torch.float32)


def _store8(x, u, keep):
    """fp32 x as E4M3 elements and a power-of-two scale for each block of 32, rounded up where the fraction and u in
    [0, 1) add up to one. keep: what is not zero stays so."""
    b = x.reshape(-1, BLOCK)
    top = b.abs().amax(1, keepdim=True)
    frac, exp = torch.frexp(top)                          # top = frac 2^exp, frac in [0.5, 1)
    e = torch.where(top > 0, torch.clamp(exp - 9 + (frac > 0.875).int(), min=-127), -127)   # top <= 448 2^e
    a = b.abs() * _power(-e)
    step = _power(torch.clamp(torch.frexp(a).exponent - 1, min=-6) - 3)
    q = torch.floor(a / step + u.reshape(-1, BLOCK)) * step
    if keep:
        q = torch.where(a > 0, torch.clamp(q, min=2.0 ** -9), q)
    code = torch.copysign(q, b).to(torch.float8_e4m3fn).reshape(-1)
    return code, (e + 127).to(torch.uint8).reshape(-1)


def _load8(code, scale):
    return (code.float().reshape(-1, BLOCK) * _power(scale.int() - 127)[:, None]).reshape(-1)


def _values8(m, ms, v, vs):
    """The 8-bit states as elements and scales: E4M3 and powers of two."""
    f8, e8 = torch.float8_e4m3fn, torch.float8_e8m0fnu
    return {"m": m.view(f8), "m_scale": ms.view(e8), "v": v.view(f8), "v_scale": vs.view(e8)}


def _plain_adamw(s):
    eight = s["bits"] == 8
    s["steps"] += 1
    t = s["steps"]
    g = s["g"].float()
    norm = None
    if s["clip"]:
        norm = torch.sqrt((g * g).sum())
        g = g * (s["max_norm"] / torch.clamp(norm, min=s["max_norm"]))
    m, v = s["m"], s["v"]
    if eight:
        m, v = _load8(m, s["m_scale"]), _load8(v, s["v_scale"]).square()
    m = B1 * m + (1 - B1) * g
    v = B2 * v + (1 - B2) * g * g
    p = s["p_flat"].float()
    p = torch.cat([p[:s["split"]] * (1 - LR * DECAY), p[s["split"]:]])
    p = p - (LR / (1 - B1 ** t)) * m / (torch.sqrt(v) * (1 - B2 ** t) ** -0.5 + ADAM_EPS)
    bits = _random(s) if eight or s["p"] == "bf16" else None
    if s["p"] == "bf16":
        whole = p.view(torch.int32) + ((bits >> 8) & 0xFFFF).int()
        s["p_flat"] = (whole & -65536).view(torch.float32).to(torch.bfloat16)
    else:
        s["p_flat"] = p
    if s["p"] == "copy":
        s["copy"] = p.to(torch.bfloat16)
    out = {"p": s["p_flat"], "copy": s["copy"], "norm": norm}
    if not eight:
        s["m"], s["v"] = m, v
        return {**out, "m": m, "v": v}
    s["m"], s["m_scale"] = _store8(m, (bits & 0xFFFF).float() / 65536, False)
    s["v"], s["v_scale"] = _store8(torch.sqrt(v), (bits >> 16).float() / 65536, True)
    return {**out, **_values8(s["m"], s["m_scale"], s["v"], s["v_scale"])}


def _dequantized(s, name, K, which):
    """fp32 [len(which), N, K] weights of the matrices `which`."""
    c, sc, z = s[name][which], s[name + "_scale"][which].float(), s[name + "_zero"][which].float()
    c = torch.stack([c & 15, c >> 4], dim=-1).flatten(-2)[..., :K].float()
    rep = lambda t: t.repeat_interleave(s["group"], dim=-1)[..., :K]  # noqa: E731
    return rep(sc) * (c - rep(z))


def _plain_w4(s):
    T, k, E, d, h = s["T"], s["k"], s["E"], s["d"], s["h"]
    flat = s["ids"].long().reshape(-1)
    some, which = torch.unique(flat, return_inverse=True)     # experts that some token picked, and which of them a slot has
    counts = torch.bincount(which)
    order = torch.sort(which, stable=True).indices
    at = torch.empty_like(order)
    at[order] = torch.arange(T * k, device=DEV) - (torch.cumsum(counts, 0) - counts)[which[order]]
    xe = torch.zeros(some.numel(), int(counts.max()), d, device=DEV)
    xe[which, at] = s["x"].float().repeat_interleave(k, dim=0)
    gate = torch.bmm(xe, _dequantized(s, "ug", d, 2 * some).transpose(1, 2))
    up = torch.bmm(xe, _dequantized(s, "ug", d, 2 * some + 1).transpose(1, 2))
    y = torch.bmm(gate / (1.0 + torch.exp(-gate)) * up, _dequantized(s, "down", h, some).transpose(1, 2))
    return (y[which, at].reshape(T, k, d) * s["weights"][:, :, None]).sum(1).to(torch.bfloat16)


def _plain_matvec(s):
    return (s["x"].float() @ _dequantized(s, "w", s["K"], torch.zeros(1, dtype=torch.int64, device=DEV))[0].T).to(torch.bfloat16)


_plain = {"join": _plain_join, "adamw": _plain_adamw, "w4": _plain_w4, "matvec": _plain_matvec}


# ----------------------------------------------------------------------------- work, and 64 bits
def _weight_bytes(group):
    return 0.5 + 2.5 / group   # half a byte, and of each group a bf16 scale and a 4-bit zero point


def work(case):
    op = case["op"]
    if op == "join":
        T, d = case["T"], case["d"]
        bx, by = (2 if case[n] == "bf16" else 4 for n in ("stream", "branch"))
        pre = case["pre"] != "none"
        if not case["backward"]:
            return {"bytes": T * d * (2 * bx + (2 if pre else 1) * by), "flops": T * d * 16}
        # dr, dx, y and dy; with a norm behind it r and dn
        return {"bytes": T * d * (2 * bx + 2 * by + (bx + by if pre else 0)) + 16 * T, "flops": T * d * 30}
    if op == "adamw":
        n = sum(map(sum, _sizes(case)))
        weight = {"fp32": 8, "copy": 10, "bf16": 4}[case["p"]]
        state = 16 if case["bits"] == 32 else 4 + 4 / BLOCK
        return {"bytes": n * (weight + state + (2 if case["g"] == "bf16" else 4)), "flops": n * 16}
    if op == "matvec":
        T, N, K = case["T"], case["N"], case["K"]
        return {"bytes": N * K * _weight_bytes(case["group"]) + 2 * T * (N + K), "flops": 2.0 * T * N * K}
    T, E, k, d, h = (case[n] for n in ("T", "E", "k", "d", "h"))
    used = E * (1 - (1 - k / E) ** T)  # experts that some token picked, on average over even picks
    return {"bytes": used * 3 * h * d * _weight_bytes(case["group"]) + 4 * T * d + 8 * T * k, "flops": 6.0 * T * k * d * h}


def exact(case, seed):
    return {"join": _exact_join, "adamw": _exact_adamw, "w4": _exact_w4, "matvec": _exact_matvec}[case["op"]](prepare(case, seed))


def _exact_norm(kind, t, gamma, beta):
    if kind == "none":
        return t
    if kind == "layer":
        var, mean = torch.var_mean(t, dim=1, unbiased=False, keepdim=True)
        t = (t - mean) / torch.sqrt(var + EPS)
    else:
        t = t / torch.sqrt((t ** 2).mean(1, keepdim=True) + EPS)
    t = t * gamma
    return t if beta is None else t + beta


def _exact_join(s):
    """The gradients by autograd from the forward's definition, in pieces of rows."""
    wide = {n: None if s[n] is None else s[n].double().requires_grad_(s["backward"])
            for n in ("post_gamma", "post_beta", "gate_w", "pre_gamma", "pre_beta")}
    gate = lambda: BRANCH if wide["gate_w"] is None else BRANCH * wide["gate_w"]  # noqa: E731
    if not s["backward"]:
        r = RES * s["x"].double() + gate() * _exact_norm(s["post"], s["y"].double(), wide["post_gamma"], wide["post_beta"])
        if s["pre"] == "none":
            return {"r": r, "n": None}
        # n is the norm of the rows as they are stored
        return {"r": r, "n": _exact_norm(s["pre"], r.to(s["x"].dtype).double(), wide["pre_gamma"], wide["pre_beta"])}
    dx, dy = torch.empty(s["r"].shape, dtype=torch.float64, device=DEV), torch.empty(s["r"].shape, dtype=torch.float64, device=DEV)
    for i in range(0, s["T"], 4096):
        rows = slice(i, i + 4096)
        r, y = s["r"][rows].double().requires_grad_(True), s["y"][rows].double().requires_grad_(True)
        D = s["dr"][rows].double()
        if s["pre"] != "none":
            n = _exact_norm(s["pre"], r, wide["pre_gamma"], wide["pre_beta"])
            n.backward(s["dn"][rows].double())
            D = D + r.grad
        (gate() * _exact_norm(s["post"], y, wide["post_gamma"], wide["post_beta"])).backward(D)
        dx[rows], dy[rows] = RES * D, y.grad
    return {"dx": dx, "dy": dy, **{"d_" + n: None if w is None else w.grad for n, w in wide.items()}}


def _exact_power(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_round(a, u, digits, lowest):
    """Non-negative a to `digits` bits after the leading one (of exponents below `lowest`: as at that one), up where the
    fraction and u add up to one."""
    e = torch.clamp(torch.frexp(a).exponent - 1, min=lowest)
    q = _exact_power(e - digits)
    return torch.floor(a / q + u) * q


def _exact_store8(x, u, keep):
    b, u = x.reshape(-1, BLOCK), u.reshape(-1, BLOCK)
    top = b.abs().amax(1, keepdim=True)
    e = torch.where(top > 0, torch.ceil(torch.log2(torch.where(top > 0, top, 1.0) / 448)), -127.0)
    e = torch.where((top > 0) & (top > 448 * _exact_power(e)), e + 1, e)        # log2 next to a power of two
    e = torch.clamp(torch.where((top > 0) & (top <= 448 * _exact_power(e - 1)), e - 1, e), min=-127.0)
    a = b.abs() / _exact_power(e)
    q = _exact_round(a, u, 3, -6)
    if keep:
        q = torch.where((a > 0) & (q == 0), 2.0 ** -9, q)
    return (torch.sign(b) * q).reshape(-1), _exact_power(e).reshape(-1)


def _exact_adamw(s):
    eight, t = s["bits"] == 8, DONE + 1
    g, norm = s["g"].double(), None
    if s["clip"]:
        norm = torch.linalg.vector_norm(g)
        g = g * min(1.0, s["max_norm"] / float(norm))
    wide = lambda c, sc: (c.double().reshape(-1, BLOCK) * _exact_power(sc.long() - 127)[:, None]).reshape(-1)  # noqa: E731
    m = torch.lerp(g, wide(s["m"], s["m_scale"]) if eight else s["m"].double(), B1)
    v = torch.lerp(g ** 2, wide(s["v"], s["v_scale"]) ** 2 if eight else s["v"].double(), B2)
    p = s["p_flat"].double()
    p[:s["split"]] -= LR * DECAY * p[:s["split"]]
    p -= LR * (m / (1 - B1 ** t)) / (torch.sqrt(v / (1 - B2 ** t)) + ADAM_EPS)
    s["steps"] = t
    bits = _random(s).double() if eight or s["p"] == "bf16" else None
    if s["p"] == "bf16":
        middle = torch.floor(bits / 256) % 65536 / 65536
        p = torch.sign(p) * _exact_round(p.abs(), middle, 7, -126)
    out = {"p": p, "copy": p if s["p"] == "copy" else None, "norm": norm}
    if not eight:
        return {**out, "m": m, "v": v}
    out["m"], out["m_scale"] = _exact_store8(m, bits % 65536 / 65536, False)
    out["v"], out["v_scale"] = _exact_store8(torch.sqrt(v), torch.floor(bits / 65536) / 65536, True)
    return out


def _exact_weight(s, name, e, K):
    c = s[name][e]
    w = torch.empty(c.shape[0], 2 * c.shape[1], dtype=torch.float64, device=DEV)
    w[:, 0::2], w[:, 1::2] = (c % 16).double(), (c // 16).double()
    w = w[:, :K]
    of = torch.arange(K, device=DEV) // s["group"]
    return (w - s[name + "_zero"][e].double()[:, of]) * s[name + "_scale"][e].double()[:, of]


def _exact_w4(s):
    out = torch.zeros(s["T"], s["d"], dtype=torch.float64, device=DEV)
    ids, w, x = s["ids"].long(), s["weights"].double(), s["x"].double()
    for e in torch.unique(ids).tolist():
        t, j = torch.nonzero(ids == e, as_tuple=True)
        a = torch.nn.functional.silu(x[t] @ _exact_weight(s, "ug", 2 * e, s["d"]).T) * (x[t] @ _exact_weight(s, "ug", 2 * e + 1, s["d"]).T)
        out.index_add_(0, t, (a @ _exact_weight(s, "down", e, s["h"]).T) * w[t, j][:, None])
    return out


def _exact_matvec(s):
    return s["x"].double() @ _exact_weight(s, "w", 0, s["K"]).T
