"""What the decode step of the 4-bit integer experts loses between its two products: SwiGLU's output reaches the down product as a
sum of two bf16 values, off by at most half a step of the second, 2^-16 of it. The rest of the tolerance is that of
test_gpu_w4.py: sums of K exact terms in fp32 units of 2^-23, K / 8 + 64 of them of the sum of the magnitudes, 64 more for SwiGLU, and
one rounding of the output."""
import numpy as np
import pytest
import torch

from oracle import train_oracle as R
from ragged_grouped_gemm_device_gb300 import _lib
from ragged_grouped_gemm_device_gb300.layer import Int4ExpertLayer
from rounding import within_one_rounding

U = 2.0 ** -23


def _weights(matrices, N, K, group, seed):
    rng = np.random.default_rng([matrices, N, K, group, seed])
    groups = (K + group - 1) // group
    codes = rng.integers(0, 16, (matrices, N, K)).astype(np.uint8)
    scales = R.to_bf16(((0.5 + rng.random((matrices, N, groups))) * K ** -0.5 / 4).astype(np.float32))
    zeros = rng.integers(0, 16, (matrices, N, groups)).astype(np.uint8)
    return (codes, scales, zeros), R.dequantize4(codes, scales, zeros, group)


def _problem(T, E, k, d, h, group):
    ug, wug = _weights(2 * E, h, d, group, 0)
    down, wd = _weights(E, d, h, group, 1)
    g = torch.Generator().manual_seed(T * 1000 + E)
    x = torch.randn(T, d, generator=g).bfloat16()
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32)
    weights = torch.rand(T, k, generator=g)
    return ug, down, wug[0::2], wug[1::2], wd, x, ids, weights


def _tolerance(d, h, mag, amag):
    return (d / 8 + 64) * U * amag + (2.0 ** -16 + (h / 8 + 128) * U) * mag


def test_one_bf16_would_not_do():
    """The tolerance tells: with SwiGLU's output rounded to one bf16 the reference itself is outside of it, with two inside."""
    T, E, k, d, h, group = 6, 4, 2, 128, 768, 32
    _, _, gate, up, wd, x, ids, weights = _problem(T, E, k, d, h, group)
    xs = x.double().numpy()
    ref, mag, amag = R.swiglu4(xs, ids.numpy(), weights.double().numpy(), gate, up, wd)
    out = np.zeros((2,) + ref.shape)
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            g = gate[e] @ xs[t]
            a = (g / (1 + np.exp(-g)) * (up[e] @ xs[t])).astype(np.float32)
            hi = R.to_bf16(a)
            lo = R.to_bf16(a - hi)
            for i, v in enumerate((hi.astype(np.float64), hi.astype(np.float64) + lo)):
                out[i, t] += float(weights[t, j]) * (wd[e] @ v)
    rounded = R.to_bf16(out.astype(np.float32)).astype(np.float64)
    assert not within_one_rounding(rounded[0], ref, _tolerance(d, h, mag, amag), torch.bfloat16)
    assert within_one_rounding(rounded[1], ref, _tolerance(d, h, mag, amag), torch.bfloat16)


# down product token by token; a block a tile for one token's slots; lists of tasks with groups of 8 and of 16, x in one and
# several segments, rows whose width is no multiple of 8
@pytest.mark.gpu
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T,E,k,d,h", [(1, 16, 8, 256, 768), (1, 5, 1, 64, 77), (1, 40, 32, 96, 100), (16, 32, 8, 128, 768), (9, 8, 4, 136, 301),
                                       (48, 4, 4, 128, 512), (60, 3, 2, 72, 133), (12, 6, 2, 64, 2200), (40, 3, 1, 64, 4300)])
def test_decode(lib, T, E, k, d, h, group):
    ug, down, gate, up, wd, x, ids, weights = _problem(T, E, k, d, h, group)
    dev = lambda c, s, z: (torch.from_numpy(R.two_to_a_byte(c)).cuda(), torch.from_numpy(s).bfloat16().cuda(), torch.from_numpy(z).cuda())
    layer = Int4ExpertLayer.from_checkpoint(dev(*ug), dev(*down), E, d, h, group)
    ref, mag, amag = R.swiglu4(x.double().numpy(), ids.numpy(), weights.double().numpy(), gate, up, wd)
    x, ids, weights = x.cuda(), ids.cuda(), weights.cuda()
    layer._buffers(T, k)
    layer.ws.fill_(255)
    out = layer.forward(x, ids, weights).clone()
    assert within_one_rounding(out.double().cpu().numpy(), ref, _tolerance(d, h, mag, amag), torch.bfloat16)
    # the output's own rounding is all that is left: half a step of 2^-8 at most
    assert np.linalg.norm(out.double().cpu().numpy() - ref) <= 2.0 ** -8 * np.linalg.norm(ref)
    layer.ws.fill_(255)
    assert torch.equal(out, layer.forward(x, ids, weights))
