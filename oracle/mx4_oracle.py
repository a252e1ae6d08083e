"""CPU fp64 reference of MXFP4 (OCP Microscaling: E2M1 elements, an E8M0 scale per 32) and of the
grouped SwiGLU forward on it."""
from __future__ import annotations

import numpy as np

BLOCK = 32
MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantize(v):
    """[..., K] -> (codes uint8 [..., K] in 0..15, scale codes uint8 [..., K / 32])."""
    v = np.asarray(v, np.float64)
    b = v.reshape(*v.shape[:-1], v.shape[-1] // BLOCK, BLOCK)
    bad = ~np.isfinite(b).all(axis=-1)
    b = np.where(bad[..., None], 0.0, b)
    top = np.abs(b).max(axis=-1)
    s = np.where(top > 0, np.maximum(np.frexp(np.where(top > 0, top, 1.0))[1] - 1 - 2, -127), -127)
    a = np.abs(b) / np.exp2(s.astype(np.float64))[..., None]
    # nearest magnitude, ties to the even code
    gap = np.abs(a[..., None] - MAGNITUDES)
    near = gap.argmin(axis=-1)
    up = np.minimum(near + 1, 7)
    tie = (np.take_along_axis(gap, near[..., None], -1) == np.take_along_axis(gap, up[..., None], -1))[..., 0]
    near = np.where(tie & (up != near) & (near % 2 == 1), up, near)
    codes = (near + 8 * np.signbit(b)).astype(np.uint8)
    scale = np.where(bad, 255, s + 127).astype(np.uint8)
    return codes.reshape(v.shape), scale


def values(codes, scale):
    """What codes and scale codes stand for; NaN where the scale is 255."""
    b = codes.reshape(*codes.shape[:-1], codes.shape[-1] // BLOCK, BLOCK)
    x = np.where(scale == 255, np.nan, np.exp2(np.minimum(scale, 254).astype(np.float64) - 127.0))
    v = MAGNITUDES[b & 7] * np.where(b & 8, -1.0, 1.0) * x[..., None]
    return v.reshape(codes.shape)


def fake_quant(v):
    return values(*quantize(v))


def swiglu_rows(xq, w_ug_q):
    """A = SwiGLU(x W_ug^T) of one expert's quantized operands (values), in fp64."""
    u = xq @ w_ug_q.T
    h = u.shape[1] // 2
    g = u[:, :h]
    return g / (1.0 + np.exp(-g)) * u[:, h:]
