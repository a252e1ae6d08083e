"""MXFP4 quantization bit for bit, and the grouped forward stage by stage: the 4-bit codes of the
SwiGLU output are read back from the workspace and checked against the fp64 values (a code may differ
only where the value lies on a rounding boundary to within the product's error), then y against the exact
product of those codes.

Tolerance of a product: E2M1 products are exact in fp32, and each of the K / 64 steps adds into an
accumulator that truncates, at most 2^-23 of the running sum of magnitudes a step and a few units
inside one: K <= 2176 here, 34 steps, so 2^-16 of the sum of magnitudes. y is one bf16 rounding of that."""
import numpy as np
import pytest
import torch

from oracle import moe_oracle as O
from oracle import mx4_oracle as Q
from ragged_grouped_gemm_device_gb300 import _lib
from rounding import within_one_rounding

pytestmark = pytest.mark.gpu
PROD = 2.0 ** -16


def _host(t):
    return t.detach().double().cpu().numpy()


def _u8(n, fill=0xFF):
    return torch.full((max(1, n),), fill, dtype=torch.uint8, device="cuda")


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


def _tiles(offsets):
    """(tile, row in tile) of every row of the problem list."""
    starts = np.concatenate([[0], offsets[:-1]])
    first = np.concatenate([[0], np.cumsum((offsets - starts + 127) // 128)[:-1]])
    p = np.arange(offsets[-1])
    e = np.searchsorted(offsets, p, side="right")
    return first[e] + (p - starts[e]) // 128, (p - starts[e]) % 128


def _unpack(q, K):
    """codes [rows, K / 2] bytes -> [rows, K] codes 0..15, the even element in the low half."""
    q = np.asarray(q).reshape(-1, K // 2)
    return np.stack([q & 15, q >> 4], axis=-1).reshape(-1, K)


def _scales(sf, G, r, K):
    """Scale codes [rows, K / 32] from the atoms, and those of the padding blocks."""
    kc = 2 * -(-K // 256)
    b = np.arange(4 * kc)
    at = (G[:, None] * kc + b // 4) * 512 + (r[:, None] % 32) * 16 + (r[:, None] // 32) * 4 + b % 4
    s = np.asarray(sf)[at]
    return s[:, : K // 32], s[:, K // 32:]


def _special(x):
    """Rows that hold zeros, subnormals, extremes, NaN and infinities."""
    K = x.shape[1]
    x[0] = 0.0
    x[1, :32] = torch.arange(32) / 4.0                       # quarter steps: ties of every kind
    if x.shape[0] > 4:
        x[2, K - 1] = 3.3e38
        x[3, 0] = 1e-39                                        # a bf16 subnormal
        x[3, 1:32] = 0.0
        x[4, 5] = float("nan")
        x[4, K - 1] = float("-inf")
    return x


@pytest.mark.parametrize("counts", [[1], [5], [128], [127, 0, 129, 3], [0, 0, 7], [200] * 3 + [0] * 297])
@pytest.mark.parametrize("K", [32, 96, 128, 160, 256, 288, 1024, 2080])
def test_rows_bit_for_bit_and_back(lib, counts, K):
    offsets = np.cumsum(counts)
    M, cap, E = int(offsets[-1]), int(offsets[-1]) + 3, len(counts)
    g = torch.Generator().manual_seed(K + M)
    x = (torch.randn(cap, K, generator=g) * torch.exp(2 * torch.randn(cap, 1, generator=g)))
    x = (_special(x) if cap > 1 else x).to(torch.bfloat16).cuda()
    q = _u8(cap * (K // 2), 0x77).view(cap, K // 2)
    sf = _u8(_lib.moe_workspace_bytes(_lib.OP_MX4_ROW_SCALES, cap, 1, E, K, 32))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    off = _i32(offsets)
    _lib.moe_mx4_quantize_rows(x, off, E, cap, K, q, sf, status)
    back = torch.full_like(x, 5.0)
    _lib.moe_mx4_dequantize_rows(q, sf, off, E, cap, K, back, status)
    torch.cuda.synchronize()
    assert status.item() == 0
    codes, scale = Q.quantize(_host(x)[:M])
    G, r = _tiles(offsets)
    got_s, pad = _scales(sf.cpu().numpy(), G, r, K)
    got_c = _unpack(q.cpu().numpy()[:M], K)
    live = np.repeat(scale != 255, 32, axis=1)               # the codes under a NaN scale carry nothing
    assert np.array_equal(got_s, scale) and (pad == 127).all()
    assert np.array_equal(got_c[live], codes[live])
    want = Q.values(codes, scale)
    b = _host(back)
    assert np.array_equal(np.nan_to_num(b[:M], nan=-9.0), np.nan_to_num(want, nan=-9.0))
    assert (b[M:] == 5.0).all() and (q[M:] == 0x77).all()    # rows past M are not written


@pytest.mark.parametrize("T,k,E,d", [(1, 1, 1, 32), (1, 8, 16, 2048), (37, 3, 5, 96), (300, 2, 4, 288), (64, 32, 40, 160)])
def test_permute_is_the_gather_quantized(lib, T, k, E, d):
    rng = np.random.default_rng(T + d)
    ids = rng.integers(-1, E, size=(T, k)).astype(np.int32)
    ids[0, 0] = 0
    r = O.route_offsets(ids, E)
    x = torch.from_numpy(rng.standard_normal((T, d)).astype(np.float32)).to(torch.bfloat16).cuda()
    n, M = T * k, r["M"]
    off, inv = _i32(r["offsets"]), _i32(r["inv_map"])
    size = _lib.moe_workspace_bytes(_lib.OP_MX4_ROW_SCALES, T, k, E, d, 32)
    q, sf, q2, sf2 = _u8(n * d // 2, 0), _u8(size, 0), _u8(n * d // 2, 0), _u8(size, 0)
    _lib.moe_permute_mxfp4(x, inv, off, T, k, E, d, q, sf)
    src = torch.from_numpy(np.asarray(r["sorted_src"][:M], np.int64) // k).cuda()
    xp = torch.zeros(n, d, dtype=torch.bfloat16, device="cuda")
    xp[:M] = x[src]
    _lib.moe_mx4_quantize_rows(xp, off, E, n, d, q2, sf2)
    torch.cuda.synchronize()
    assert torch.equal(q, q2) and torch.equal(sf, sf2)


@pytest.mark.parametrize("K", [32, 160, 288, 1056, 2080])
def test_many_rows_bit_for_bit_and_back(lib, K):
    """Rows enough that a warp takes 1024 elements at a time; special values in every part of a row."""
    offsets = np.cumsum([1000, 0, 1601])
    M, cap = int(offsets[-1]), int(offsets[-1]) + 2
    g = torch.Generator().manual_seed(K)
    x = torch.randn(cap, K, generator=g) * torch.exp(2 * torch.randn(cap, 1, generator=g))
    x[3::11] *= 2.0 ** -127                                  # subnormal and tiny normal values
    x[4::11] *= 2.0 ** 120
    x[5::11, K - 1] = float("nan")
    x[6::11, K // 2] = float("inf")
    x[7::11, : K // 2] = 0.0
    x = x.clamp(-3.3e38, 3.3e38).where(~x.isinf(), x).to(torch.bfloat16).cuda()
    q = _u8(cap * (K // 2), 0x77).view(cap, K // 2)
    sf = _u8(_lib.moe_workspace_bytes(_lib.OP_MX4_ROW_SCALES, cap, 1, 3, K, 32))
    off = _i32(offsets)
    _lib.moe_mx4_quantize_rows(x, off, 3, cap, K, q, sf)
    back = torch.full_like(x, 5.0)
    _lib.moe_mx4_dequantize_rows(q, sf, off, 3, cap, K, back)
    torch.cuda.synchronize()
    codes, scale = Q.quantize(_host(x)[:M])
    assert (scale == 0).any() and (scale == 255).any() and (scale > 240).any()
    G, r = _tiles(offsets)
    got_s, pad = _scales(sf.cpu().numpy(), G, r, K)
    live = np.repeat(scale != 255, 32, axis=1)
    assert np.array_equal(got_s, scale) and (pad == 127).all()
    assert np.array_equal(_unpack(q.cpu().numpy()[:M], K)[live], codes[live])
    b = _host(back)
    assert np.array_equal(np.nan_to_num(b[:M], nan=-9.0), np.nan_to_num(Q.values(codes, scale), nan=-9.0))
    assert (b[M:] == 5.0).all() and (q[M:] == 0x77).all()


@pytest.mark.parametrize("T,k,E,d", [(2500, 3, 5, 96), (2431, 1, 2, 1056), (2600, 8, 16, 288)])
def test_permute_of_many_tokens(lib, T, k, E, d):
    test_permute_is_the_gather_quantized(lib, T, k, E, d)


def test_weights_of_many_rows(lib):
    test_weights_bit_for_bit(lib, 5, 1056, 256)


def _prepared(w_ug, w_down):
    E, h2, d = w_ug.shape
    h = h2 // 2
    mxw = _u8(_lib.moe_workspace_bytes(_lib.OP_MX4_WEIGHTS, 0, 1, E, d, h))
    _lib.moe_mx4_prepare_weights(w_ug, w_down, E, d, h, mxw)
    return mxw


@pytest.mark.parametrize("E,d,h", [(1, 32, 32), (3, 96, 160), (2, 256, 128), (2, 288, 416)])
def test_weights_bit_for_bit(lib, E, d, h):
    g = torch.Generator().manual_seed(d + h)
    w_ug = torch.randn(E, 2 * h, d, generator=g).to(torch.bfloat16).cuda()
    w_down = torch.randn(E, h, d, generator=g).to(torch.bfloat16).cuda()
    raw = _prepared(w_ug, w_down).cpu().numpy()
    r256 = lambda b: (b + 255) // 256 * 256
    at = 0
    for w, K, N, per in ((_host(w_ug).reshape(E * 2, h, d), d, h, -(-h // 128)),
                         (_host(w_down).transpose(0, 2, 1), h, d, 2 * -(-(-(-d // 128)) // 2))):
        groups = w.shape[0]
        codes, scale = Q.quantize(w)
        nq = groups * N * K // 2
        assert np.array_equal(_unpack(raw[at:at + nq], K), codes.reshape(-1, K))
        at += r256(nq)
        n = np.arange(N)
        G = (np.arange(groups)[:, None] * per + n // 128).reshape(-1)
        ns = groups * per * 2 * -(-K // 256) * 512
        s, pad = _scales(raw[at:at + ns], G, np.tile(n % 128, groups), K)
        assert np.array_equal(s, scale.reshape(-1, K // 32)) and (pad == 127).all()
        at += r256(ns)
    assert at == raw.size


# counts around the 128-row tiles, empty experts, one expert, many; widths that end inside a stage of
# 256, a 128-row weight tile and a 256-column tile; an odd number of 128-element chunks of h
CASES = [([1], 32, 32), ([3], 256, 128), ([1, 0, 2, 1], 288, 96), ([127, 0, 129, 5], 160, 416), ([128, 256], 512, 256),
         ([0, 0, 300, 0], 1056, 160), ([2] * 40, 96, 544), ([0] * 5 + [1] + [0] * 290, 2048, 768), ([700, 9], 128, 2176),
         ([16] * 8, 2048, 512), ([40, 8, 0, 33, 64, 65], 640, 384)]


@pytest.mark.parametrize("counts,d,h", CASES)
def test_forward(lib, counts, d, h):
    E, offsets = len(counts), np.cumsum(counts)
    M, cap = int(offsets[-1]), int(offsets[-1]) + 130
    g = torch.Generator().manual_seed(M + d + h)
    used = [e for e in range(E) if counts[e]]
    w_ug = torch.full((E, 2 * h, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    w_down = torch.full((E, h, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    for e in used:  # an expert without rows is not read
        w_ug[e] = (torch.randn(2 * h, d, generator=g) / d ** 0.5).to(torch.bfloat16)
        w_down[e] = (torch.randn(h, d, generator=g) / h ** 0.5).to(torch.bfloat16)
    mxw = _prepared(w_ug, w_down)
    x = torch.randn(cap, d, generator=g).to(torch.bfloat16).cuda()
    x[M:] = float("nan")
    off = _i32(offsets)
    q = _u8(cap * d // 2).view(cap, d // 2)
    sf = _u8(_lib.moe_workspace_bytes(_lib.OP_MX4_ROW_SCALES, cap, 1, E, d, h))
    ws = _u8(_lib.moe_workspace_bytes(_lib.OP_MX4_FWD, cap, 1, E, d, h))
    y = torch.full((cap, d), 3.0, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    _lib.moe_mx4_quantize_rows(x, off, E, cap, d, q, sf, status)
    _lib.moe_grouped_swiglu_fwd_mxfp4(q, sf, off, E, cap, d, h, mxw, y, ws, status)
    torch.cuda.synchronize()
    assert status.item() == 0
    again = torch.empty_like(y)
    _lib.moe_grouped_swiglu_fwd_mxfp4(q, sf, off, E, cap, d, h, mxw, again, ws, status)
    got, raw = _host(y), ws.cpu().numpy()
    assert torch.equal(again[:M], y[:M]) and (got[M:] == 3.0).all()
    G, r = _tiles(offsets)
    a_codes = _unpack(raw[: M * h // 2], h)
    nq = (cap * h // 2 + 255) // 256 * 256
    a_scale, pad = _scales(raw[nq:], G, r, h)
    assert (pad == 127).all()
    a_val = Q.values(a_codes, a_scale)
    for e in used:
        rows = slice(offsets[e] - counts[e], offsets[e])
        xq = Q.fake_quant(_host(x[rows]))
        wu, wd = Q.fake_quant(_host(w_ug[e])), Q.fake_quant(_host(w_down[e]).T)
        u, mag = xq @ wu.T, np.abs(xq) @ np.abs(wu).T
        gate, up = u[:, :h], u[:, h:]
        s = 1.0 / (1.0 + np.exp(-gate))
        a = gate * s * up
        # error of A: the products' errors through silu (|silu'| <= 1.1) and the multiplication, and
        # the approximate exponential and division (|gate| + 4 units of 2^-23)
        err = (1.1 * PROD * mag[:, :h] * np.abs(up) + np.abs(gate * s) * PROD * mag[:, h:]
               + (np.abs(gate) + 4) * 2.0 ** -23 * np.abs(a))
        block = a.reshape(len(a), -1, 32)
        eb = err.reshape(block.shape)
        scale = np.exp2(a_scale[rows].astype(np.float64) - 127)[..., None]
        vals = a_val[rows].reshape(block.shape)
        # the block's exponent is that of its maximum, which may lie within its error of a power of two
        top, te = np.abs(block).max(-1), eb.max(-1)
        lo, hi = np.maximum(top - te, 1e-300), top + te
        want_lo, want_hi = np.floor(np.log2(lo)) - 2, np.floor(np.log2(hi)) - 2
        s_code = a_scale[rows].astype(np.float64) - 127
        assert ((s_code >= np.maximum(want_lo, -127)) & (s_code <= np.maximum(want_hi, -127))).all()
        # the value stored is the quantization of some value within the error: monotone rounding
        def quant(v):
            t = np.abs(v) / scale
            idx = np.minimum((t[..., None] > np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])).sum(-1), 7)
            return np.sign(v) * Q.MAGNITUDES[idx] * scale
        step = 1e-12 * scale  # ties themselves may go either way by the error's edge
        assert ((vals >= quant(block - eb - step)) & (vals <= quant(block + eb + step))).all()
        # y from the codes the kernel stored
        ref, m2 = a_val[rows] @ wd.T, np.abs(a_val[rows]) @ np.abs(wd).T
        assert within_one_rounding(got[rows], ref, PROD * m2, torch.bfloat16)


def test_a_nan_stays_in_its_row(lib):
    E, d, h, M = 2, 512, 256, 70
    g = torch.Generator().manual_seed(5)
    w_ug = (torch.randn(E, 2 * h, d, generator=g) / d ** 0.5).to(torch.bfloat16).cuda()
    w_down = (torch.randn(E, h, d, generator=g) / h ** 0.5).to(torch.bfloat16).cuda()
    mxw, off = _prepared(w_ug, w_down), _i32([40, 70])
    x = torch.randn(M, d, generator=g).to(torch.bfloat16).cuda()

    def run(x):
        q = _u8(M * d // 2).view(M, d // 2)
        sf = _u8(_lib.moe_workspace_bytes(_lib.OP_MX4_ROW_SCALES, M, 1, E, d, h))
        ws = _u8(_lib.moe_workspace_bytes(_lib.OP_MX4_FWD, M, 1, E, d, h))
        y = torch.zeros(M, d, dtype=torch.bfloat16, device="cuda")
        _lib.moe_mx4_quantize_rows(x, off, E, M, d, q, sf)
        _lib.moe_grouped_swiglu_fwd_mxfp4(q, sf, off, E, M, d, h, mxw, y, ws)
        return y

    clean = run(x)
    x[3, 100], x[50, 511] = float("nan"), float("inf")
    got = run(x)
    rest = [t for t in range(M) if t not in (3, 50)]
    assert torch.isnan(got[[3, 50]]).all() and torch.equal(got[rest], clean[rest])


def test_bad_offsets_write_nothing(lib):
    E, d, h, cap = 3, 64, 64, 20
    mxw = _prepared(torch.zeros(E, 2 * h, d, dtype=torch.bfloat16, device="cuda"),
                    torch.zeros(E, h, d, dtype=torch.bfloat16, device="cuda"))
    for bad in ([5, 3, 20], [5, 10, 21], [-1, 4, 9]):
        off = _i32(bad)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        q = _u8(cap * d // 2, 9).view(cap, d // 2)
        sf = _u8(_lib.moe_workspace_bytes(_lib.OP_MX4_ROW_SCALES, cap, 1, E, d, h), 9)
        x = torch.ones(cap, d, dtype=torch.bfloat16, device="cuda")
        _lib.moe_mx4_quantize_rows(x, off, E, cap, d, q, sf, status)
        assert status.item() == _lib.MOE_DEV_BAD_OFFSETS and (q == 9).all() and (sf == 9).all()
        status.zero_()
        ws = _u8(_lib.moe_workspace_bytes(_lib.OP_MX4_FWD, cap, 1, E, d, h))
        y = torch.full((cap, d), 3.0, dtype=torch.bfloat16, device="cuda")
        _lib.moe_grouped_swiglu_fwd_mxfp4(q, sf, off, E, cap, d, h, mxw, y, ws, status)
        assert status.item() == _lib.MOE_DEV_BAD_OFFSETS and (y == 3.0).all()
