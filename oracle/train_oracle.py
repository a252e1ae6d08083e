"""CPU fp64 references of what trains and serves a block: the residual join of two norms, AdamW with its 8-bit states, and
4-bit integer weights with group scales."""
from __future__ import annotations

import numpy as np

BLOCK = 32


# ------------------------------------------------------------------------------------------- residual join
def norm(kind, v, eps):
    """(normalised rows, mean, rstd) of v [T, d]."""
    T = v.shape[0]
    mean = v.mean(axis=1) if kind == "layer" else np.zeros(T)
    if kind == "none":
        return v, mean, np.ones(T)
    c = v - mean[:, None]
    rstd = 1.0 / np.sqrt((c * c).mean(axis=1) + eps)
    return c * rstd[:, None], mean, rstd


def _w(w, fill):
    return fill if w is None else np.asarray(w, np.float64)


def join(x, y, post, post_gamma, post_beta, gate, res_scale, branch_scale, eps):
    """r (not rounded) of x [T, d] and y [T, d] or None; (r, yhat, mean, rstd)."""
    x = np.asarray(x, np.float64)
    if y is None:
        return res_scale * x, np.zeros_like(x), np.zeros(x.shape[0]), np.ones(x.shape[0])
    yhat, mean, rstd = norm(post, np.asarray(y, np.float64), eps)
    z = yhat * _w(post_gamma, 1.0) + _w(post_beta, 0.0)
    return res_scale * x + branch_scale * _w(gate, 1.0) * z, yhat, mean, rstd


def norm_grad(kind, g, hat, rstd):
    """The gradient of the rows from g, the gradient of the normalised rows."""
    if kind == "none":
        return g
    out = g - hat * (g * hat).mean(axis=1, keepdims=True)
    if kind == "layer":
        out = out - g.mean(axis=1, keepdims=True)
    return out * rstd[:, None]


def join_grad(dn, dr, r, y, post, post_gamma, post_beta, gate, pre, pre_gamma, res_scale, branch_scale, eps):
    """A dict of every gradient, D (that of r), and yhat, rhat with their rstd."""
    r = None if r is None else np.asarray(r, np.float64)
    shape = next(np.asarray(t).shape for t in (dr, dn) if t is not None)
    D = np.zeros(shape) if dr is None else np.asarray(dr, np.float64).copy()
    o = {}
    if pre != "none":
        dn = np.asarray(dn, np.float64)
        o["rhat"], _, o["rstd2"] = norm(pre, r, eps)
        o["g2"] = dn * _w(pre_gamma, 1.0)
        D = D + norm_grad(pre, o["g2"], o["rhat"], o["rstd2"])
        o["d_pre_gamma"], o["d_pre_beta"] = (dn * o["rhat"]).sum(axis=0), dn.sum(axis=0)
    o["D"], o["dx"] = D, res_scale * D
    if y is not None:
        o["yhat"], _, o["rstd1"] = norm(post, np.asarray(y, np.float64), eps)
        dz = branch_scale * _w(gate, 1.0) * D
        o["d_gate"] = (branch_scale * D * (o["yhat"] * _w(post_gamma, 1.0) + _w(post_beta, 0.0))).sum(axis=0)
        o["d_post_gamma"], o["d_post_beta"] = (dz * o["yhat"]).sum(axis=0), dz.sum(axis=0)
        o["g1"] = dz * _w(post_gamma, 1.0)
        o["dy"] = norm_grad(post, o["g1"], o["yhat"], o["rstd1"])
    return o


# ------------------------------------------------------------------------------------------- AdamW
def mix(x):
    """The finalizer of MurmurHash3 on uint32 values."""
    x = np.asarray(x, np.uint64) & np.uint64(0xFFFFFFFF)
    m = np.uint64(0xFFFFFFFF)
    x = ((x ^ (x >> np.uint64(16))) * np.uint64(0x85EBCA6B)) & m
    x = ((x ^ (x >> np.uint64(13))) * np.uint64(0xC2B2AE35)) & m
    return x ^ (x >> np.uint64(16))


def random_bits(seed, t, tensor, n):
    key = mix(np.uint64(seed) ^ mix((0x9E3779B9 * t + tensor) & 0xFFFFFFFF))
    i = np.arange(n, dtype=np.uint64)
    return mix(key + (i & np.uint64(0xFFFFFFFF)) * np.uint64(0x9E3779B9) + (i >> np.uint64(32)) * np.uint64(0x85EBCA6B))


def round_up_where(a, u, digits, lowest):
    """a >= 0 to `digits` bits after the leading one (below 2^lowest: the steps there), up where the fraction and u in [0, 1)
    reach 1. Returns (value, step, distance of fraction + u from the next whole number that decides)."""
    e = np.maximum(np.frexp(np.where(a > 0, a, 1.0))[1] - 1, lowest)
    step = np.ldexp(1.0, e - digits)
    s = a / step + u
    return np.floor(s) * step, step, np.abs(s - np.round(s))


def scale_exponent(x):
    """s of each block of 32: the smallest, not below -127, with max |x| <= 448 * 2^s (-127 for a block of zeros)."""
    top = np.abs(_blocks(x)).max(axis=1)
    frac, e = np.frexp(top)
    return np.where(top > 0, np.maximum(e - 9 + (frac > 0.875), -127), -127)


def _blocks(x):
    n = (x.size + BLOCK - 1) // BLOCK * BLOCK
    return np.concatenate([x, np.zeros(n - x.size)]).reshape(-1, BLOCK)


def quantize8(x, u, keep):
    """(elements in units of their scale, scale exponents, distance from the threshold) of x [n] in blocks of 32."""
    s = scale_exponent(x)
    b, ub = _blocks(x), _blocks(u)
    a = np.abs(b) / np.ldexp(1.0, s)[:, None]
    q, _, far = round_up_where(a, ub, 3, -6)
    if keep:
        q = np.where(a > 0, np.maximum(q, 2.0 ** -9), q)
    return (np.sign(b) * q).reshape(-1)[:x.size], s, far.reshape(-1)[:x.size]


def adamw(p, g, m, v, t, lr, beta1, beta2, eps, decay, c=1.0):
    """(p, m, v) after step t (from 1), in fp64, not rounded."""
    g = c * np.asarray(g, np.float64)
    m = beta1 * np.asarray(m, np.float64) + (1 - beta1) * g
    v = beta2 * np.asarray(v, np.float64) + (1 - beta2) * g * g
    up = (m / (1 - beta1 ** t)) / (np.sqrt(v / (1 - beta2 ** t)) + eps)
    return np.asarray(p, np.float64) * (1 - lr * decay) - lr * up, m, v


# ------------------------------------------------------------------------------------------- 4-bit integers
def to_bf16(a):
    """fp32 values rounded to the nearest bf16, ties to even (finite values)."""
    u = np.asarray(a, np.float32).view(np.uint32).astype(np.uint64)
    u = (u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000
    return u.astype(np.uint32).view(np.float32)


def quantize4(w, group):
    """(codes, scales, zeros) of bf16 rows w [rows, K]: codes [rows, K] one to a byte, in fp32 arithmetic as specified."""
    rows, K = w.shape
    groups = (K + group - 1) // group
    codes, scales, zeros = np.zeros((rows, K), np.uint8), np.zeros((rows, groups), np.float32), np.zeros((rows, groups), np.uint8)
    f = np.float32
    for j in range(groups):
        b = np.asarray(w[:, j * group:(j + 1) * group], np.float32)
        lo, hi = np.minimum(b.min(axis=1), f(0)), np.maximum(b.max(axis=1), f(0))
        s = to_bf16(hi / f(15) - lo / f(15))
        safe = np.where(s > 0, s, f(1))
        z = np.where(s > 0, np.clip(np.rint(-lo / safe), 0, 15), 0).astype(np.float32)
        c = np.clip(np.rint(b / safe[:, None]) + z[:, None], 0, 15)
        codes[:, j * group:(j + 1) * group] = np.where(s[:, None] > 0, c, 0)
        scales[:, j], zeros[:, j] = s, z
    return codes, scales, zeros


def two_to_a_byte(codes):
    c = np.concatenate([codes, np.zeros(codes.shape[:-1] + (codes.shape[-1] % 2,), np.uint8)], axis=-1)
    return c[..., 0::2] | (c[..., 1::2] << 4)


def dequantize4(codes, scales, zeros, group):
    """fp64 weights of codes [..., K], scales and zeros [..., groups] (zeros None: 8)."""
    of = np.arange(codes.shape[-1]) // group
    z = 8.0 if zeros is None else np.asarray(zeros, np.float64)[..., of]
    return np.asarray(scales, np.float64)[..., of] * (codes.astype(np.float64) - z)


def pack4(codes, scales_bits, zeros, group):
    """The packed bytes of codes [matrices, N, K] (one to a byte), bf16 scale bits and zeros [matrices, N, groups], element by
    element from the layout's description."""
    M, N, K = codes.shape
    tiles, chunks, per = (N + 15) // 16, (K + 127) // 128, 128 // group
    size = (1024 + 40 * per + 15) // 16 * 16
    out = np.zeros((M * tiles * chunks * size + 255) // 256 * 256, np.uint8)
    place = [0, 2, 4, 6, 1, 3, 5, 7]   # the element whose code each nibble holds
    for m in range(M):
        for tile in range(tiles):
            for chunk in range(chunks):
                base = ((m * tiles + tile) * chunks + chunk) * size
                for r in range(16):
                    row = tile * 16 + r
                    if row >= N:
                        continue
                    for q in range(4):
                        for t in range(4):
                            word = 0
                            for nib in range(8):
                                k = chunk * 128 + 32 * q + 8 * t + place[nib]
                                first = chunk * 128 + 32 * q + 8 * t
                                if first >= K:
                                    continue
                                c = int(codes[m, row, k]) if k < K else int(zeros[m, row, first // group])
                                word |= c << (4 * nib)
                            word = (word << 3 | word >> 29) & 0xFFFFFFFF
                            at = base + (r // 8) * 512 + ((r % 8) * 4 + t) * 16 + 4 * q
                            out[at:at + 4] = np.frombuffer(np.uint32(word).tobytes(), np.uint8)
                    for j in range(per):
                        gj = chunk * per + j
                        if gj * group >= K:
                            continue
                        at = base + 1024 + ((r % 8) * per + j) * 4 + (r // 8) * 2
                        out[at:at + 2] = np.frombuffer(np.uint16(scales_bits[m, row, gj]).tobytes(), np.uint8)
                        out[base + 1024 + 32 * per + (r % 8) * per + j] |= np.uint8(int(zeros[m, row, gj]) << (4 * (r // 8)))
    return out


def swiglu4(x, ids, weights, gate, up, down):
    """out [T, d] of dequantized experts: gate, up [E, h, d], down [E, d, h] (fp64), SwiGLU's output rounded to bf16; and the sum of the
    magnitudes of its terms."""
    T, k = ids.shape
    E = gate.shape[0]
    out, mag, amag = np.zeros((T, down.shape[1])), np.zeros((T, down.shape[1])), np.zeros((T, down.shape[1]))
    for t in range(T):
        for j in range(k):
            e = ids[t, j]
            if not 0 <= e < E:
                continue
            w = 1.0 if weights is None else float(weights[t, j])
            g, u = gate[e] @ x[t], up[e] @ x[t]
            s = 1.0 / (1.0 + np.exp(-g))
            a = g * s * u
            # what an error of one part of the sums of |w x| does to a
            ag, au = np.abs(gate[e]) @ np.abs(x[t]), np.abs(up[e]) @ np.abs(x[t])
            da = np.abs(u) * (s * (1 + np.abs(g) * (1 - s))) * ag + np.abs(g * s) * au
            out[t] += w * (down[e] @ a)
            mag[t] += abs(w) * (np.abs(down[e]) @ np.abs(a))
            amag[t] += abs(w) * (np.abs(down[e]) @ da)
    return out, mag, amag
