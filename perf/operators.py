"""Cases of the operators around and inside the mixture-of-experts block, with their plain forms.

Three operators that a mixture-of-experts block needs next to the grouped expert products:

* ``layer_norm``  -- the block's pre-norm: layer norm over the last dimension, forward and
                     backward, with the gradients of its weight and bias.
* ``gate``        -- the router: softmax over the experts, the top_k experts per token with their
                     weights, per-expert counts, the balance and z losses, and their gradient.
* ``mx4_*``       -- MXFP4 (4-bit E2M1 elements, one power-of-two scale per 32): quantising rows
                     and reading them back, and the SwiGLU experts with both operands of every
                     product in MXFP4, from token rows to combined token rows.

``run`` computes them in their plain form (elementary torch operations in 32 bits, rounded once)
unless ``own`` is true, when it makes the library's calls.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
BLOCK = 32           # elements per MXFP4 scale
RENORM = 1           # gate flag: weights normalised over the selected experts
EPS = 1e-5
LARGEST_NORM = 16384 * 2048      # elements of the largest layer norm case
LARGEST_GATE = 131072 * 256      # logits of the largest gate case
LARGEST_TRIP = 131072 * 2048     # elements of the largest round trip
LARGEST_FWD = 131072 * 2048 * 512  # rows * d * h of the largest expert forward


def listed():
    return [
        # pre-norm of a decode step: 16 sequences, one token each; latency
        dict(name="norm decode", op="layer_norm", T=16, d=2048, dtype="bf16", backward=False),
        # pre-norm of one training step of the large workload
        dict(name="norm train large", op="layer_norm", T=16384, d=2048, dtype="bf16", backward=True),
        # fp32 activations, row and width that fill no tile (the skew workload's sizes)
        dict(name="norm train odd fp32", op="layer_norm", T=20000, d=1000, dtype="fp32", backward=True),
        # routing one decode step of the fine-grained workload: ids and weights only
        dict(name="gate decode", op="gate", T=16, E=128, k=8, dtype="bf16", renorm=True, masked=0.0, backward=False),
        # router of one fine-grained training step: fp32 logits, losses and gradient
        dict(name="gate train finegrained", op="gate", T=4096, E=128, k=8, dtype="fp32", renorm=True, masked=0.0,
             backward=True),
        # eight times the large workload's tokens, a tenth of them padding; full-softmax weights
        dict(name="gate train large masked", op="gate", T=131072, E=256, k=8, dtype="bf16", renorm=False, masked=0.1,
             backward=True),
        # a prompt of 333 tokens as it enters a 4-bit layer
        dict(name="mx4 trip small", op="mx4_trip", M=333, K=1024),
        # the gathered rows of the large workload
        dict(name="mx4 trip large", op="mx4_trip", M=131072, K=2048),
        # one token through the 4-bit fine-grained layer
        dict(name="mx4 one token", op="mx4_fwd", T=1, E=128, k=8, d=2048, h=768, skew=0.5),
        # one decode step of 16 sequences
        dict(name="mx4 decode", op="mx4_fwd", T=16, E=128, k=8, d=2048, h=768, skew=0.5),
        # prefill of the fine-grained layer
        dict(name="mx4 prefill finegrained", op="mx4_fwd", T=4096, E=128, k=8, d=2048, h=768,
             skew=0.5),
        # prefill at the large workload's sizes
        dict(name="mx4 prefill large", op="mx4_fwd", T=16384, E=256, k=8, d=2048, h=512,
             skew=0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["layer_norm", "gate", "mx4_trip", "mx4_fwd"])
    if op == "layer_norm":
        d = _log(rng, 64, 8192)
        d += d == 3072
        if rng.random() < 0.5:
            d = max(64, d // 64 * 64) + 64 * (d // 64 * 64 == 3072)
        return dict(op=op, T=_log(rng, 1, min(32768, LARGEST_NORM // d)), d=d, dtype=rng.choice(["bf16", "fp32"]),
                    backward=rng.random() < 0.7)
    if op == "gate":
        E = _log(rng, 4, 512)
        return dict(op=op, T=_log(rng, 1, min(131072, LARGEST_GATE // E)), E=E, k=rng.randint(1, min(E, 8)),
                    dtype=rng.choice(["bf16", "fp32"]), renorm=rng.random() < 0.5, masked=rng.choice([0.0, 0.1, 0.4]),
                    backward=rng.random() < 0.7)
    if op == "mx4_trip":
        K = BLOCK * _log(rng, 4, 256)
        K += BLOCK * (K == 3072)
        return dict(op=op, M=_log(rng, 1, min(131072, LARGEST_TRIP // K)), K=K)
    E, k = _log(rng, 4, 256), rng.randint(1, 8)
    k = min(k, E)
    d, h = BLOCK * _log(rng, 8, 80), BLOCK * _log(rng, 8, 64)
    while E * d * h > 256 * 2048 * 512:
        E = max(k, E // 2)
        if E == k:
            break
    return dict(op=op, T=_log(rng, 1, min(16384, max(1, LARGEST_FWD // (d * h * k)))), E=E, k=k, d=d, h=h,
                skew=rng.choice([0.0, 0.5]))


# ------------------------------------------------------------------------------------- inputs
_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _normal(g, *shape, dtype=torch.float32, std=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * std).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = dict(case)
    op = case["op"]
    if op == "layer_norm":
        T, d, t = case["T"], case["d"], _TYPES[case["dtype"]]
        # residual stream: a per-channel offset and spread, weights near one
        spread = torch.exp(0.3 * _normal(g, d))
        s["x"] = (_normal(g, T, d) * spread + 0.3 * _normal(g, d)).to(t)
        s["gamma"], s["beta"] = 1.0 + 0.2 * _normal(g, d), 0.1 * _normal(g, d)
        s["dy"] = _normal(g, T, d, dtype=t)
    elif op == "gate":
        T, E, k, t = case["T"], case["E"], case["k"], _TYPES[case["dtype"]]
        # N(0, 1) logits with a per-expert bias, which skews the load mildly
        s["logits"] = (_normal(g, T, E) + 0.5 * _normal(g, E)).to(t)
        s["mask"] = torch.rand(T, generator=g, device=DEV) >= case["masked"] if case["masked"] > 0 else None
        s["d_weights"] = _normal(g, T, k)
        s["d_loss"] = torch.tensor([0.01 * T, 0.001 * T], device=DEV) * (0.5 + torch.rand(2, generator=g, device=DEV))
    elif op == "mx4_trip":
        M, K = case["M"], case["K"]
        s["x"] = (_normal(g, M, K) * torch.exp(0.5 * _normal(g, K))).to(torch.bfloat16)
        s["offsets"] = torch.tensor([M], dtype=torch.int32, device=DEV)
    else:
        T, E, k, d, h = (case[n] for n in ("T", "E", "k", "d", "h"))
        s["x"] = (_normal(g, T, d) * torch.exp(0.5 * _normal(g, d))).to(torch.bfloat16)
        # the weights as a 4-bit checkpoint holds them: the values their codes and scales stand for
        s["w_ug"] = torch.empty(E, 2 * h, d, dtype=torch.bfloat16, device=DEV)
        s["w_down"] = torch.empty(E, h, d, dtype=torch.bfloat16, device=DEV)
        step = max(1, (1 << 26) // (2 * h * d))
        for e in range(0, E, step):
            n = min(step, E - e)
            s["w_ug"][e:e + n] = _fake_quant(_normal(g, n, 2 * h, d, std=d ** -0.5))
            s["w_down"][e:e + n] = _fake_quant(_normal(g, n, d, h, std=h ** -0.5)).transpose(1, 2)
        # the routing of this batch, as the router and moe_route_offsets leave it
        logits = _normal(g, T, E) + s["skew"] * _normal(g, E)
        top = torch.sort(logits, dim=1, descending=True, stable=True)
        ids = top.indices[:, :k]
        s["ids"] = ids.to(torch.int32).contiguous()
        s["weights"] = torch.softmax(top.values[:, :k], dim=1).contiguous()
        order = torch.sort(ids.reshape(-1), stable=True).indices
        s["sorted_src"] = order.to(torch.int32)
        inv = torch.empty_like(order)
        inv[order] = torch.arange(T * k, device=DEV)
        s["inv_map"] = inv.to(torch.int32)
        s["offsets"] = torch.cumsum(torch.bincount(ids.reshape(-1), minlength=E), 0).to(torch.int32)
    if own:
        _buffers(s)
    return s


def _buffers(s):
    """The output and work buffers a user's program keeps, and the weights laid out once."""
    from ragged_grouped_gemm_device_gb300 import _lib as L
    f32, i32, u8 = torch.float32, torch.int32, torch.uint8
    new = lambda *shape, dtype=f32: torch.empty(*shape, dtype=dtype, device=DEV)  # noqa: E731
    room = lambda *a: new(max(1, L.moe_workspace_bytes(*a)), dtype=u8)  # noqa: E731
    op = s["op"]
    if op == "layer_norm":
        T, d = s["T"], s["d"]
        s["y"], s["mean"], s["rstd"] = torch.empty_like(s["x"]), new(T), new(T)
        if s["backward"]:
            s["dx"], s["dgamma"], s["dbeta"] = torch.empty_like(s["x"]), new(d), new(d)
            s["ws"] = room(L.OP_LAYER_NORM_BWD, T, 1, 1, d)
    elif op == "gate":
        T, E, k = s["T"], s["E"], s["k"]
        s["ids"], s["weights"], s["lse"] = new(T, k, dtype=i32), new(T, k), new(T)
        s["mask8"] = None if s["mask"] is None else s["mask"].view(u8)
        if s["backward"]:
            s["counts"], s["n_valid"], s["prob_sum"], s["loss"] = new(E, dtype=i32), new(1, dtype=i32), new(E), new(2)
            s["dlogits"] = torch.empty_like(s["logits"])
            s["ws"] = room(L.OP_GATE, T, k, E)
    elif op == "mx4_trip":
        M, K = s["M"], s["K"]
        s["q"] = new(M, K // 2, dtype=u8)
        s["sf"] = room(L.OP_MX4_ROW_SCALES, M, 1, 1, K, 32)
        s["back"] = torch.empty_like(s["x"])
    else:
        T, E, k, d, h = (s[n] for n in ("T", "E", "k", "d", "h"))
        s["mxw"] = room(L.OP_MX4_WEIGHTS, 0, 1, E, d, h)
        L.moe_mx4_prepare_weights(s["w_ug"], s["w_down"], E, d, h, s["mxw"])
        s["xq"] = new(T * k, d // 2, dtype=u8)
        s["xsf"] = room(L.OP_MX4_ROW_SCALES, T, k, E, d, h)
        s["ws"] = room(L.OP_MX4_FWD, T, k, E, d, h)
        s["y"] = new(T * k, d, dtype=torch.bfloat16)
        s["out"] = torch.empty_like(s["x"])


# ------------------------------------------------------------------------------- the operators
def run(s):
    return (_own if own else _plain)[s["op"]](s)


def _own_layer_norm(s):
    from ragged_grouped_gemm_device_gb300 import _lib as L
    T, d = s["T"], s["d"]
    if not s["backward"]:
        L.moe_layer_norm_fwd(s["x"], s["gamma"], s["beta"], T, d, EPS, s["y"])
        return {"y": s["y"]}
    L.moe_layer_norm_fwd(s["x"], s["gamma"], s["beta"], T, d, EPS, s["y"], s["mean"], s["rstd"])
    L.moe_layer_norm_bwd(s["dy"], s["x"], s["gamma"], s["mean"], s["rstd"], T, d, s["dx"], s["dgamma"], s["dbeta"],
                         s["ws"])
    return {n: s[n] for n in ("y", "dx", "dgamma", "dbeta")}


def _own_gate(s):
    from ragged_grouped_gemm_device_gb300 import _lib as L
    T, E, k = s["T"], s["E"], s["k"]
    flags = RENORM if s["renorm"] else 0
    if not s["backward"]:
        L.moe_gate_fwd(s["logits"], s["mask8"], T, k, E, flags, s["ids"], s["weights"])
        return {"ids": s["ids"], "weights": s["weights"]}
    L.moe_gate_fwd(s["logits"], s["mask8"], T, k, E, flags, s["ids"], s["weights"], s["lse"], s["counts"],
                   s["n_valid"], s["prob_sum"], s["loss"], s["ws"])
    L.moe_gate_bwd(s["logits"], s["lse"], s["ids"], s["weights"], s["counts"], s["n_valid"], s["d_weights"],
                   s["d_loss"], T, k, E, flags, s["dlogits"])
    return {n: s[n] for n in ("ids", "weights", "counts", "prob_sum", "loss", "dlogits")}


def _own_mx4_trip(s):
    from ragged_grouped_gemm_device_gb300 import _lib as L
    L.moe_mx4_quantize_rows(s["x"], s["offsets"], 1, s["M"], s["K"], s["q"], s["sf"])
    L.moe_mx4_dequantize_rows(s["q"], s["sf"], s["offsets"], 1, s["M"], s["K"], s["back"])
    return s["back"]


def _own_mx4_fwd(s):
    from ragged_grouped_gemm_device_gb300 import _lib as L
    T, E, k, d, h = (s[n] for n in ("T", "E", "k", "d", "h"))
    L.moe_permute_mxfp4(s["x"], s["inv_map"], s["offsets"], T, k, E, d, s["xq"], s["xsf"])
    L.moe_grouped_swiglu_fwd_mxfp4(s["xq"], s["xsf"], s["offsets"], E, T * k, d, h, s["mxw"], s["y"], s["ws"])
    L.moe_unpermute_combine(s["y"], s["inv_map"], s["weights"], T, k, d, s["out"])
    return s["out"]


_own = {"layer_norm": _own_layer_norm, "gate": _own_gate, "mx4_trip": _own_mx4_trip, "mx4_fwd": _own_mx4_fwd}


def _plain_layer_norm(s):
    x = s["x"].float()
    mean = x.mean(1, keepdim=True)
    c = x - mean
    rstd = torch.rsqrt((c * c).mean(1, keepdim=True) + EPS)
    xhat = c * rstd
    y = (xhat * s["gamma"] + s["beta"]).to(s["x"].dtype)
    if not s["backward"]:
        return {"y": y}
    dy = s["dy"].float()
    gdy = dy * s["gamma"]
    dx = rstd * (gdy - gdy.mean(1, keepdim=True) - xhat * (gdy * xhat).mean(1, keepdim=True))
    return {"y": y, "dx": dx.to(s["x"].dtype), "dgamma": (dy * xhat).sum(0), "dbeta": dy.sum(0)}


def _plain_gate(s):
    E, k = s["E"], s["k"]
    lg = s["logits"].float()
    m = lg.amax(1, keepdim=True)
    e = torch.exp(lg - m)
    total = e.sum(1, keepdim=True)
    p = e / total
    lse = (m + torch.log(total)).squeeze(1)
    ids = torch.sort(lg, dim=1, descending=True, stable=True).indices[:, :k]
    w = torch.gather(p, 1, ids)
    picked = w.sum(1, keepdim=True)
    if s["renorm"]:
        w = w / picked
    on = torch.ones(lg.shape[0], dtype=torch.bool, device=lg.device) if s["mask"] is None else s["mask"]
    live = on[:, None]
    ids_out = torch.where(live, ids, -1).to(torch.int32)
    w = torch.where(live, w, 0.0)
    if not s["backward"]:
        return {"ids": ids_out, "weights": w}
    p = torch.where(live, p, 0.0)
    n = on.sum().float()
    counts = torch.zeros(E + 1, dtype=torch.int32, device=lg.device)
    counts.index_add_(0, torch.where(live, ids, E).reshape(-1), torch.ones(ids.numel(), dtype=torch.int32, device=lg.device))
    counts = counts[:E]
    prob_sum = p.sum(0)
    share = counts.float() / torch.clamp(n * k, min=1.0)
    per = 1.0 / torch.clamp(n, min=1.0)
    balance = E * (share * prob_sum).sum() * per
    z = (torch.where(on, lse, 0.0) ** 2).sum() * per
    # d(loss)/dp, then through the softmax; the z loss adds 2 lse p / n
    dw = torch.where(live, s["d_weights"], 0.0)
    dp = (s["d_loss"][0] * E * per * share).expand_as(p)
    dlogits = p * (2.0 * s["d_loss"][1] * per * lse)[:, None]
    if s["renorm"]:
        sel = w * (dw - (w * dw).sum(1, keepdim=True))
    else:
        sel = torch.zeros_like(w)
        dp = dp.scatter_add(1, ids, dw)
    dlogits = dlogits + p * (dp - (p * dp).sum(1, keepdim=True))
    dlogits = dlogits.scatter_add(1, ids, sel)
    dlogits = torch.where(live, dlogits, 0.0)
    return {"ids": ids_out, "weights": w, "counts": counts, "prob_sum": prob_sum, "loss": torch.stack([balance, z]),
            "dlogits": dlogits.to(s["logits"].dtype)}


def _fake_quant(x):
    """The values the MXFP4 codes of fp32 rows stand for, block by block along the last dimension."""
    b = x.reshape(*x.shape[:-1], -1, BLOCK)
    amax = b.abs().amax(-1, keepdim=True)
    s = torch.where(amax > 0, torch.clamp(torch.frexp(amax).exponent - 3, min=-127), -127)
    inv = ((127 - s) << 23).view(torch.float32)
    v = b * inv
    a = v.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    a = torch.clamp(torch.round(a / step) * step, max=6.0)
    return (torch.copysign(a, v) / inv).reshape(x.shape)


def _plain_mx4_trip(s):
    return _fake_quant(s["x"].float()).to(torch.bfloat16)


def _plain_mx4_fwd(s):
    T, E, k, h = s["T"], s["E"], s["k"], s["h"]
    src = s["sorted_src"].long()
    expert = s["ids"].reshape(-1).long()[src]                 # of each row in expert order
    counts = torch.bincount(expert, minlength=E)
    some = torch.nonzero(counts).squeeze(1)                   # experts with rows
    place = torch.cumsum(counts > 0, 0) - 1
    first = torch.cumsum(counts, 0) - counts
    at = torch.arange(T * k, device=src.device) - first[expert]
    rows = int(counts.max())
    xe = torch.zeros(some.numel(), rows, s["d"], device=src.device)
    xe[place[expert], at] = _fake_quant(s["x"].float())[src // k]
    u = torch.bmm(xe, s["w_ug"][some].float().transpose(1, 2))
    gate, up = u[..., :h], u[..., h:]
    a = _fake_quant(gate / (1.0 + torch.exp(-gate)) * up)
    y = torch.bmm(a, s["w_down"][some].float())[place[expert], at]
    w = s["weights"].unsqueeze(2)
    return (y[s["inv_map"].long()].reshape(T, k, -1) * w).sum(1).to(torch.bfloat16)


_plain = {"layer_norm": _plain_layer_norm, "gate": _plain_gate, "mx4_trip": _plain_mx4_trip, "mx4_fwd": _plain_mx4_fwd}


# ----------------------------------------------------------------------------- work, and 64 bits
def work(case):
    op = case["op"]
    es = {"bf16": 2, "fp32": 4}.get(case.get("dtype"), 2)
    if op == "layer_norm":
        T, d = case["T"], case["d"]
        # x (and dy) in, y (and dx) out; the weight, bias and their gradients
        n = 4 if case["backward"] else 2
        return {"bytes": T * d * es * n + 4 * d * n, "flops": T * d * (8 + (13 if case["backward"] else 0))}
    if op == "gate":
        T, E, k = case["T"], case["E"], case["k"]
        out = T * k * 8
        if not case["backward"]:
            return {"bytes": T * E * es + out, "flops": T * E * 5}
        return {"bytes": 2 * T * E * es + out + T * k * 4 + E * 8, "flops": T * E * 11}
    if op == "mx4_trip":
        # bf16 in and out; codes (half a byte) and scales (1/32 byte) written and read back
        n = case["M"] * case["K"]
        return {"bytes": n * 4 + 2 * n * (0.5 + 1 / BLOCK), "flops": n * 4}
    T, E, k, d, h = (case[n] for n in ("T", "E", "k", "d", "h"))
    used = E * (1 - (1 - k / E) ** T)  # experts that some token picked, on average over even picks
    return {"bytes": 2 * 2 * T * d + used * 3 * h * d * (0.5 + 1 / BLOCK) + 8 * T * k, "flops": 6.0 * T * k * d * h}


def exact(case, seed):
    s = prepare(case, seed)
    return _exact[case["op"]](s)


def _exact_layer_norm(s):
    x, g = s["x"].double(), s["gamma"].double()
    var, mean = torch.var_mean(x, dim=1, unbiased=False, keepdim=True)
    z = (x - mean) / torch.sqrt(var + EPS)
    y = z * g + s["beta"].double()
    if not s["backward"]:
        return {"y": y}
    dy, d = s["dy"].double(), x.shape[1]
    dz = dy * g
    dx = (d * dz - dz.sum(1, keepdim=True) - z * (dz * z).sum(1, keepdim=True)) / (d * torch.sqrt(var + EPS))
    return {"y": y, "dx": dx, "dgamma": torch.einsum("td,td->d", dy, z), "dbeta": dy.sum(0)}


def _exact_gate(s):
    E, k = s["E"], s["k"]
    rows = torch.arange(s["T"], device=DEV) if s["mask"] is None else torch.nonzero(s["mask"]).squeeze(1)
    lg = s["logits"][rows].double().requires_grad_(True)
    pick = torch.argsort(-lg.detach(), dim=1, stable=True)[:, :k]
    w = torch.softmax(lg, 1).gather(1, pick)
    if s["renorm"]:
        w = torch.softmax(lg.gather(1, pick), 1)

    def spread(v, dtype=torch.float64, fill=0.0):
        full = torch.full((s["T"], v.shape[1]), fill, dtype=dtype, device=DEV)
        full[rows] = v.to(dtype)
        return full

    ids, weights = spread(pick, torch.int32, -1), spread(w.detach())
    if not s["backward"]:
        return {"ids": ids, "weights": weights}
    n = max(1, rows.numel())
    counts = torch.bincount(pick.reshape(-1), minlength=E)
    prob = torch.softmax(lg, 1).sum(0)
    loss = torch.stack([E * (counts / (n * k) * prob / n).sum(), torch.logsumexp(lg, 1).square().sum() / n])
    whole = (w * s["d_weights"][rows].double()).sum() + (loss * s["d_loss"].double()).sum()
    grad, = torch.autograd.grad(whole, lg)
    return {"ids": ids, "weights": weights, "counts": counts.to(torch.int32), "prob_sum": prob.detach(),
            "loss": loss.detach(), "dlogits": spread(grad)}


def _exact_fake_quant(v):
    """MXFP4 by its definition in 64 bits: nearest of the eight magnitudes, ties to the even code."""
    b = v.reshape(*v.shape[:-1], -1, BLOCK)
    top = b.abs().amax(-1, keepdim=True)
    low = torch.clamp(torch.floor(torch.log2(torch.where(top > 0, top, 1.0))), min=-125.0) - 2.0
    # floor(log2) next to a power of two may be off by a rounding: mend it against the power itself
    low = torch.where(top >= torch.exp2(low + 3), low + 1, torch.where((top < torch.exp2(low + 2)) & (low > -127), low - 1, low))
    low = torch.where(top > 0, low, -127.0)
    a = (b / torch.exp2(low)).abs()
    code = sum((a > m).int() for m in (0.25, 1.25, 2.5, 5.0)) + sum((a >= m).int() for m in (0.75, 1.75, 3.5))
    mags = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device=v.device)
    return (mags[code.long()] * torch.sign(b) * torch.exp2(low)).reshape(v.shape)


def _exact_mx4_trip(s):
    step = max(1, (1 << 25) // s["K"])
    return torch.cat([_exact_fake_quant(s["x"][i:i + step].double()).float() for i in range(0, s["M"], step)])


def _exact_mx4_fwd(s):
    T, E, k, h = s["T"], s["E"], s["k"], s["h"]
    out = torch.zeros(T, s["d"], dtype=torch.float64, device=DEV)
    ids, w = s["ids"].long(), s["weights"].double()
    for e in torch.unique(ids).tolist():
        t, j = torch.nonzero(ids == e, as_tuple=True)
        u = _exact_fake_quant(s["x"][t].double()) @ s["w_ug"][e].double().T
        a = _exact_fake_quant(torch.nn.functional.silu(u[:, :h]) * u[:, h:])
        out.index_add_(0, t, (a @ s["w_down"][e].double()) * w[t, j][:, None])
    return out


_exact = {"layer_norm": _exact_layer_norm, "gate": _exact_gate, "mx4_trip": _exact_mx4_trip, "mx4_fwd": _exact_mx4_fwd}
