"""Sizes at which the kernels of layer norm, the gate and the MXFP4 experts go round their loops: more tiles than SMs,
more row pieces or tokens than warps, more rows than the ring holds and than one load of row statistics covers. The references and
tolerances are those of the smaller cases."""
import numpy as np
import pytest
import torch

import test_gpu_gate as G
import test_gpu_layer_norm as N
import test_gpu_mx4 as M
from oracle import mx4_oracle as Q
from ragged_grouped_gemm_device_gb300 import _lib

pytestmark = pytest.mark.gpu


# On 152 SMs: a CTA takes a second and third tile of both products, with several stages each; an expert has more
# row tiles than a raster group (16); tiles of few rows (the 16-row boxes) follow one another
@pytest.mark.parametrize("counts,d,h", [([2500, 0, 130, 3000], 1056, 800), ([40] * 60, 544, 416),
                                        ([2100] + [17] * 30 + [0, 129], 800, 1184)])
def test_products_of_more_tiles_than_sms(lib, counts, d, h):
    tiles = sum(-(-c // 128) for c in counts)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert tiles * -(-d // 256) > sms and tiles * -(-h // 128) > sms
    M.test_forward(lib, counts, d, h)


# a warp has a second piece from 2 x 9728 pieces on (8 blocks of 8 warps an SM)
@pytest.mark.parametrize("K", [288, 1056])
def test_rows_and_back_of_more_pieces_than_warps(lib, K):
    offsets = np.cumsum([9000, 0, 12001, 3000, 6])
    rows, E = int(offsets[-1]), 5
    cap = rows + 2
    g = torch.Generator().manual_seed(K)
    x = torch.randn(cap, K, generator=g) * torch.exp(2 * torch.randn(cap, 1, generator=g))
    x[5::1013, K - 1] = float("nan")
    x[6::1013, K // 2] = float("inf")
    x[7::1013, : K // 2] = 0.0
    x = x.to(torch.bfloat16).cuda()
    q = M._u8(cap * (K // 2), 0x77).view(cap, K // 2)
    sf = M._u8(_lib.moe_workspace_bytes(_lib.OP_MX4_ROW_SCALES, cap, 1, E, K, 32))
    off = M._i32(offsets)
    _lib.moe_mx4_quantize_rows(x, off, E, cap, K, q, sf)
    back = torch.full_like(x, 5.0)
    _lib.moe_mx4_dequantize_rows(q, sf, off, E, cap, K, back)
    torch.cuda.synchronize()
    tile, r = M._tiles(offsets)
    got_s, pad = M._scales(sf.cpu().numpy(), tile, r, K)
    got_c, b = M._unpack(q.cpu().numpy()[:rows], K), M._host(back)
    assert (pad == 127).all() and (b[rows:] == 5.0).all() and (q[rows:] == 0x77).all()
    for i in range(0, rows, 2000):
        at = slice(i, min(rows, i + 2000))
        codes, scale = Q.quantize(M._host(x[at]))
        live = np.repeat(scale != 255, 32, axis=1)
        assert np.array_equal(got_s[at], scale) and np.array_equal(got_c[at][live], codes[live])
        assert np.array_equal(np.nan_to_num(b[at], nan=-9.0), np.nan_to_num(Q.values(codes, scale), nan=-9.0))


@pytest.mark.parametrize("T,k,E,d", [(30000, 2, 5, 96), (21000, 3, 7, 1056)])
def test_permute_of_more_pieces_than_warps(lib, T, k, E, d):
    M.test_permute_is_the_gather_quantized(lib, T, k, E, d)


def test_weights_of_more_pieces_than_threads(lib):
    """All experts at once against each by itself, which is held to the definition bit for bit."""
    E, d, h = 32, 544, 1280
    M.test_weights_bit_for_bit(lib, 1, d, h)
    g = torch.Generator("cuda").manual_seed(1)
    w_ug = torch.randn(E, 2 * h, d, generator=g, device="cuda").to(torch.bfloat16)
    w_down = torch.randn(E, h, d, generator=g, device="cuda").to(torch.bfloat16)
    r256 = lambda b: (b + 255) // 256 * 256
    sizes = [2 * h * d // 2, 2 * 10 * 6 * 512, h * d // 2, 6 * 10 * 512]  # codes and atoms of an expert, W_ug and W_down
    whole = M._prepared(w_ug, w_down).cpu().numpy()
    alone = [M._prepared(w_ug[e:e + 1], w_down[e:e + 1]).cpu().numpy() for e in range(E)]
    at = part = 0
    for n in sizes:
        for e in range(E):
            assert np.array_equal(whole[at + e * n: at + (e + 1) * n], alone[e][part: part + n]), (n, e)
        at, part = at + r256(E * n), part + r256(n)
    assert at == whole.size and part == alone[0].size


# more than 32 rows a block in the backward, more than the forward's ring in each: every layout of threads a row,
# with a number of rows that the blocks do not share evenly
@pytest.mark.parametrize("dtype,T,d", [("bf16", 60001, 64), ("fp32", 59003, 128), ("bf16", 60001, 65), ("bf16", 60001, 328),
                                       ("bf16", 15001, 1032), ("fp32", 14999, 512), ("bf16", 9999, 2056),
                                       ("fp32", 9999, 1028), ("bf16", 4999, 4104), ("fp32", 4999, 4100), ("fp32", 15001, 1001)])
def test_layer_norm_of_many_rows_a_block(lib, dtype, T, d):
    x, dy, gamma, beta = N._inputs(T, d, dtype)
    N._check(x, dy, gamma, beta, N._run(x, dy, gamma, beta))


# a lane group has several tokens, in every layout of lanes and lists of both directions; E = 60 and 250 are read
# one element at a time
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,E,k,renorm", [(40003, 64, 4, True), (40003, 60, 3, False), (30001, 128, 8, True), (25001, 256, 8, False),
                                          (10007, 250, 6, True), (12001, 512, 4, True), (6007, 1000, 5, False), (6007, 1001, 5, True)])
def test_gate_of_many_tokens_a_lane_group(lib, T, E, k, renorm, dtype):
    mask = torch.rand(T, generator=torch.Generator().manual_seed(E)).cuda() > 0.1
    G.Gate(G._logits(T, E, dtype), mask, k, renorm).run().check()
