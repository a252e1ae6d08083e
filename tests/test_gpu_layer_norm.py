"""Layer norm forward and backward against the fp64 reference.

Tolerances. y and dx are a handful of fp32 roundings (unit 2^-24) of terms no larger than `scale`, plus
the error of the mean, at most (threads' tree depth + terms per thread) roundings of the row's largest
magnitude: 64 units of the terms' scale cover both; bf16 outputs are one rounding of such a value.
A weight gradient is a sum of T terms added at most T / 608 + 64 deep: each level rounds once."""
import numpy as np
import pytest
import torch

from oracle import block_oracle as B
from ragged_grouped_gemm_device_gb300 import _lib
from rounding import within_one_rounding

pytestmark = pytest.mark.gpu
U32 = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _host(t):
    return t.detach().double().cpu().numpy()


def _inputs(T, d, dtype, w_dtype="fp32", offset=0.3, seed=0):
    g = torch.Generator().manual_seed(1000 * T + d + seed)
    x = (torch.randn(T, d, generator=g) * 1.2 + offset).to(TYPES[dtype]).cuda()
    dy = torch.randn(T, d, generator=g).to(TYPES[dtype]).cuda()
    gamma = (1 + 0.2 * torch.randn(d, generator=g)).to(TYPES[w_dtype]).cuda()
    beta = (0.1 * torch.randn(d, generator=g)).to(TYPES[w_dtype]).cuda()
    return x, dy, gamma, beta


def _run(x, dy, gamma, beta, eps=1e-5, y=None, dx=None):
    T, d = x.shape
    nan = lambda *s, dtype=torch.float32: torch.full(s, float("nan"), dtype=dtype, device="cuda")
    y = nan(T, d, dtype=x.dtype) if y is None else y
    dx = nan(T, d, dtype=x.dtype) if dx is None else dx
    mean, rstd, dgamma, dbeta = nan(T), nan(T), nan(d), nan(d)
    ws = nan(max(1, _lib.moe_workspace_bytes(_lib.OP_LAYER_NORM_BWD, T, 1, 1, d) // 4))
    _lib.moe_layer_norm_fwd(x, gamma, beta, T, d, eps, y, mean, rstd)
    _lib.moe_layer_norm_bwd(dy, x, gamma, mean, rstd, T, d, dx, dgamma, dbeta, ws)
    torch.cuda.synchronize()
    return y, mean, rstd, dx, dgamma, dbeta


def _check(x, dy, gamma, beta, got, eps=1e-5):
    y, mean, rstd, dx, dgamma, dbeta = (_host(t) for t in got)
    T, d = x.shape
    xh, dyh = _host(x), _host(dy)
    g = None if gamma is None else _host(gamma)
    b = None if beta is None else _host(beta)
    ry, rm, rr, xhat = B.layer_norm(xh, g, b, eps)
    rdx, rdg, rdb = B.layer_norm_grad(dyh, xh, g, eps)
    gg = np.ones(d) if g is None else g
    big = np.abs(xh).max(axis=1)                                    # the mean's error is in units of it
    loss = (1 + big * rr)[:, None]                                   # units lost relative to rstd
    assert (np.abs(mean - rm) <= 64 * U32 * big).all()
    # the variance is a sum of squares of differences with errors of 64 units of `big`
    assert (np.abs(rstd - rr) <= 64 * U32 * rr * (1 + big * rr)).all()
    scale = (np.abs(xhat) + 1) * np.abs(gg) * loss + (0 if b is None else np.abs(b))
    assert within_one_rounding(y, ry, 64 * U32 * scale, x.dtype)
    gd = np.abs(dyh * gg)
    terms = (gd + gd.mean(axis=1, keepdims=True) + (np.abs(xhat) + 1) * (gd * (np.abs(xhat) + 1)).mean(axis=1, keepdims=True))
    assert within_one_rounding(dx, rdx, 64 * U32 * rr[:, None] * terms * loss, x.dtype)
    depth = T / 608 + 64
    assert (np.abs(dgamma - rdg) <= depth * U32 * (np.abs(dyh) * (np.abs(xhat) + 1) * loss).sum(axis=0)).all()
    assert (np.abs(dbeta - rdb) <= depth * U32 * np.abs(dyh).sum(axis=0)).all()


# widths on both sides of each register layout's limit, odd ones (one element an access), one of
# the layout without registers; row counts from one to more than the backward's blocks
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,d", [(1, 1), (1, 2048), (3, 8), (5, 31), (2, 127), (7, 256), (4, 264), (9, 512), (6, 1000),
                                 (3, 1001), (2, 2056), (3, 4096), (2, 4104), (2, 8191), (2, 8192), (1, 8200),
                                 (1, 16384), (2, 16392), (1, 40001), (700, 96), (1300, 2048), (2500, 65)])
def test_matches_the_reference(lib, T, d, dtype):
    x, dy, gamma, beta = _inputs(T, d, dtype)
    _check(x, dy, gamma, beta, _run(x, dy, gamma, beta))


@pytest.mark.parametrize("w_dtype", ["bf16", "none"])
@pytest.mark.parametrize("d", [100, 1024, 20000])
def test_bf16_and_absent_weights(lib, d, w_dtype):
    x, dy, gamma, beta = _inputs(33, d, "bf16", "bf16")
    if w_dtype == "none":
        gamma = beta = None
    _check(x, dy, gamma, beta, _run(x, dy, gamma, beta))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_rows_of_a_wider_buffer(lib, dtype):
    """Row pitches and bases that are no multiple of 16 bytes, and an upstream gradient that is one
    row for all tokens (what a sum's backward broadcasts)."""
    T, d = 19, 520
    x, dy, gamma, beta = _inputs(T, d + 11, dtype)
    xs, ys, dxs = x[:, 3:3 + d], torch.full_like(x, float("nan"))[:, 1:1 + d], torch.full_like(x, float("nan"))[:, 5:5 + d]
    one = dy[:1, 2:2 + d].expand(T, d)
    got = _run(xs, one, gamma[:d].contiguous(), beta[:d].contiguous(), y=ys, dx=dxs)
    _check(xs, one, gamma[:d], beta[:d], got)
    wide = torch.full((T, d + 16), float("nan"), dtype=x.dtype, device="cuda")
    aligned = _run(xs.contiguous(), dy[:, :d].contiguous(), gamma[:d].contiguous(), beta[:d].contiguous(), y=wide[:, 8:8 + d])
    _check(xs.contiguous(), dy[:, :d].contiguous(), gamma[:d], beta[:d], aligned)
    assert torch.isnan(wide[:, :8]).all() and torch.isnan(wide[:, 8 + d:]).all()  # nothing outside the rows


def test_large_offset_and_constant_rows(lib):
    """A mean far above the spread keeps the two-pass variance's accuracy; a constant row has
    variance 0 and gives beta."""
    x, dy, gamma, beta = _inputs(8, 768, "fp32", offset=200.0)
    _check(x, dy, gamma, beta, _run(x, dy, gamma, beta))
    x[:] = 3.0
    y = _run(x, dy, gamma, beta)[0]
    assert torch.equal(y, beta.expand_as(y))


def test_nan_and_infinity_stay_in_their_rows(lib):
    x, dy, gamma, beta = _inputs(6, 320, "bf16")
    clean = _run(x, dy, gamma, beta)
    x[2, 7], x[4, 0] = float("nan"), float("inf")
    got = _run(x, dy, gamma, beta)
    for i in (0, 3):  # y, dx
        assert torch.isnan(got[i][[2, 4]]).all()
        assert torch.equal(got[i][[0, 1, 3, 5]], clean[i][[0, 1, 3, 5]])


def test_no_rows_and_repeated_calls(lib):
    x, dy, gamma, beta = _inputs(4, 64, "bf16")
    e = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    dg, db = torch.full((64,), float("nan"), device="cuda"), torch.full((64,), float("nan"), device="cuda")
    s = torch.empty(0, device="cuda")
    _lib.moe_layer_norm_fwd(e, gamma, beta, 0, 64, 1e-5, e)
    _lib.moe_layer_norm_bwd(e, e, gamma, s, s, 0, 64, e, dg, db)
    assert (dg == 0).all() and (db == 0).all()
    x, dy, gamma, beta = _inputs(5000, 512, "bf16")
    a, b = _run(x, dy, gamma, beta), _run(x, dy, gamma, beta)
    assert all(torch.equal(p, q) for p, q in zip(a, b))  # a fixed order of every sum


def test_on_another_stream(lib):
    x, dy, gamma, beta = _inputs(64, 256, "bf16")
    want = _run(x, dy, gamma, beta)[0]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = torch.empty_like(x)
    _lib.moe_layer_norm_fwd(x, gamma, beta, 64, 256, 1e-5, y, stream=s)
    s.synchronize()
    assert torch.equal(y, want)


def test_refusals(lib):
    x, dy, gamma, beta = _inputs(4, 64, "bf16")
    y = torch.empty_like(x)
    with pytest.raises(ValueError):
        _lib.moe_layer_norm_fwd(x.t(), gamma, beta, 64, 4, 1e-5, y)          # columns are not contiguous
    with pytest.raises(ValueError):
        _lib.moe_layer_norm_fwd(x.half(), gamma, beta, 4, 64, 1e-5, y)
    with pytest.raises(ValueError):
        _lib.moe_layer_norm_fwd(x, gamma, beta.bfloat16(), 4, 64, 1e-5, y)   # weights of two types
    with pytest.raises(ValueError):
        _lib.moe_layer_norm_fwd(x, gamma[:32], beta[:32], 4, 64, 1e-5, y)
    with pytest.raises(_lib.MoEError):
        _lib.moe_layer_norm_fwd(x, gamma, beta, 4, 64, -1.0, y)
    with pytest.raises(_lib.MoEError):                                       # workspace missing
        m = torch.zeros(4, device="cuda")
        _lib.moe_layer_norm_bwd(dy, x, gamma, m, m, 4, 64, y, torch.empty(64, device="cuda"))
