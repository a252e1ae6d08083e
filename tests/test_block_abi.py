"""Host-side refusals of the layer norm, gate and MXFP4 entry points, and their workspace sizes (no GPU:
validation fails before any CUDA call)."""
import ctypes

import pytest

from ragged_grouped_gemm_device_gb300 import _lib, build

INVALID, SHAPE, WS = 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


p, p2 = ctypes.c_void_p(256), ctypes.c_void_p(258)  # never dereferenced
BIG = 1 << 30


def test_workspaces():
    build.build()
    wb = _lib.moe_workspace_bytes
    # layer norm: two fp32 partial rows for each of at most 608 blocks
    assert wb(_lib.OP_LAYER_NORM_BWD, 16384, 1, 1, 2048) == 608 * 2 * 2048 * 4
    assert wb(_lib.OP_LAYER_NORM_BWD, 5, 1, 1, 100) == 5 * 2 * 100 * 4
    assert wb(_lib.OP_LAYER_NORM_BWD, 5, 1, 1, 0) == 0 and wb(_lib.OP_LAYER_NORM_BWD, 5, 1, 1, (1 << 20) + 1) == 0
    # codes at half a byte; scale atoms: 512 bytes per 128 rows and 128 of K, chunks padded to even
    assert wb(_lib.OP_MX4_ROW_SCALES, 4096, 8, 128, 2048, 768) == (32768 + 127 * 128) // 128 * 16 * 512
    assert wb(_lib.OP_MX4_ROW_SCALES, 100, 1, 1, 288, 32) == (100 + 127) // 128 * 4 * 512
    assert wb(_lib.OP_MX4_FWD, 100, 1, 1, 64, 160) == (100 * 80 + 255) // 256 * 256 + 2 * 512
    E, d, h = 3, 288, 160
    assert wb(_lib.OP_MX4_WEIGHTS, 0, 1, E, d, h) == (E * 2 * h * d // 2 + E * 2 * 2 * 4 * 512
                                                      + E * d * h // 2 + E * 4 * 2 * 512)
    for bad in ((100, 64), (64, 100), (0, 64)):
        assert wb(_lib.OP_MX4_FWD, 4, 1, 2, *bad) == 0
    assert wb(_lib.OP_GATE, 4096, 8, 128) > 0 and wb(_lib.OP_GATE, 0, 1, 1) > 0


def test_layer_norm_refusals(lib):
    f, b = lib.moe_layer_norm_fwd, lib.moe_layer_norm_bwd
    assert f(p, 0, 64, p, p, 1, -1, 64, 1e-5, p, 64, p, p, None) == INVALID
    assert f(p, 0, 64, p, p, 1, 4, 0, 1e-5, p, 64, p, p, None) == INVALID
    assert f(p, 0, 64, p, p, 1, 4, (1 << 20) + 1, 1e-5, p, (1 << 20) + 1, p, p, None) == SHAPE
    assert f(p, 2, 64, p, p, 1, 4, 64, 1e-5, p, 64, p, p, None) == INVALID           # no such type
    assert f(p, 0, 64, p, p, 1, 4, 64, 1e-5, p, 63, p, p, None) == INVALID           # rows of y overlap
    assert f(p, 0, -64, p, p, 1, 4, 64, 1e-5, p, 64, p, p, None) == INVALID
    assert f(None, 0, 64, p, p, 1, 4, 64, 1e-5, p, 64, p, p, None) == INVALID
    assert f(p2, 1, 64, p, p, 1, 4, 64, 1e-5, p, 64, p, p, None) == INVALID          # fp32 at 2 mod 4
    for eps in (-1.0, float("nan"), float("inf")):
        assert f(p, 0, 64, p, p, 1, 4, 64, eps, p, 64, p, p, None) == INVALID
    assert b(p, 64, p, 64, 0, p, 1, p, p, 4, 64, p, 64, p, p, None, 0, None) == WS
    assert b(p, 64, p, 64, 0, p, 1, p, p, 4, 64, p, 64, p, p, p, 4 * 2 * 64 * 4 - 1, None) == WS
    assert b(p, 64, p, 64, 0, p, 1, None, p, 4, 64, p, 64, p, p, p, BIG, None) == INVALID
    assert b(p, 64, p, 64, 0, p, 1, p, p, 4, 64, p, 60, p, p, p, BIG, None) == INVALID


def test_gate_refusals(lib):
    f, b = lib.moe_gate_fwd, lib.moe_gate_bwd
    none = (None, None, None, None)
    assert f(p, 0, 8, None, 4, 9, 8, 0, p, p, p, *none, None, 0, None) == SHAPE      # top_k > E
    assert f(p, 0, 64, None, 4, 33, 64, 0, p, p, p, *none, None, 0, None) == SHAPE
    assert f(p, 0, 2000, None, 4, 2, 2000, 0, p, p, p, *none, None, 0, None) == SHAPE
    assert f(p, 0, 8, None, 1 << 30, 2, 8, 0, p, p, p, *none, None, 0, None) == SHAPE
    assert f(p, 0, 8, None, -1, 2, 8, 0, p, p, p, *none, None, 0, None) == INVALID
    assert f(p, 3, 8, None, 4, 2, 8, 0, p, p, p, *none, None, 0, None) == INVALID
    assert f(p, 0, 8, None, 4, 2, 8, 4, p, p, p, *none, None, 0, None) == INVALID    # unknown flag
    assert f(p, 0, 8, None, 4, 2, 8, 0, None, p, p, *none, None, 0, None) == INVALID
    assert f(p, 0, 8, None, 4, 2, 8, 0, p, p, p, p, p, p, None, p, BIG, None) == INVALID  # statistics in part
    assert f(p, 0, 8, None, 4, 2, 8, 0, p, p, p, p, p, p, p, None, 0, None) == WS
    assert b(p, 0, 8, p, p, p, p, p, p, p, 4, 2, 8, 0, p, 7, None) == INVALID        # rows of dlogits overlap
    assert b(p, 0, 8, None, p, p, p, p, p, p, 4, 2, 8, 0, p, 8, None) == INVALID
    assert b(p, 0, 8, p, None, p, p, p, p, p, 4, 2, 8, 0, p, 8, None) == INVALID     # d_weights without ids
    assert b(p, 0, 8, p, p, p, None, p, p, p, 4, 2, 8, 0, p, 8, None) == INVALID     # d_loss without counts


def test_mx4_refusals(lib):
    fwd = lambda E, cap, d, h, mxw=p, ws=p, n=BIG: lib.moe_grouped_swiglu_fwd_mxfp4(p, p, p, E, cap, d, h, mxw, p, ws, n, None, None)
    assert fwd(4, 10, 48, 64) == SHAPE and fwd(4, 10, 64, 80) == SHAPE and fwd(1025, 10, 64, 64) == SHAPE
    assert fwd(4, -1, 64, 64) == INVALID and fwd(0, 10, 64, 64) == INVALID
    assert fwd(4, 10, 64, 64, mxw=p2) == INVALID and fwd(4, 10, 64, 64, ws=p2) == INVALID
    assert fwd(4, 10, 64, 64, n=_lib.moe_workspace_bytes(_lib.OP_MX4_FWD, 10, 1, 4, 64, 64) - 1) == WS
    assert fwd(1, (1 << 31) - 128, 1 << 20, 32) == SHAPE                             # tiles beyond an int
    assert lib.moe_mx4_prepare_weights(p, p, 4, 64, 64, p, 16, None) == WS
    assert lib.moe_mx4_prepare_weights(p, p, 4, 64, 33, p, BIG, None) == SHAPE
    assert lib.moe_mx4_quantize_rows(p, p, 4, 10, 40, p, p, None, None) == SHAPE
    assert lib.moe_mx4_quantize_rows(p, None, 4, 10, 64, p, p, None, None) == INVALID
    assert lib.moe_mx4_dequantize_rows(p, p, p, 4, 10, 40, p, None, None) == SHAPE
    assert lib.moe_mx4_dequantize_rows(p, p, p, 4, 10, 64, p2, None, None) == INVALID
    assert lib.moe_permute_mxfp4(p, p, p, 10, 2, 4, 40, p, p, None, None) == SHAPE
    assert lib.moe_permute_mxfp4(p, p, p, 10, 33, 4, 64, p, p, None, None) == SHAPE
    assert lib.moe_permute_mxfp4(p, None, p, 10, 2, 4, 64, p, p, None, None) == INVALID
