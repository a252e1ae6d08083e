"""4-bit integer weights with group scales against the fp64 reference.

Tolerances. Codes, scales and the packed layout are exact. A product's fp32 sum of K exact terms, in any order and with sums
that truncate (unit 2^-23), is off by at most K / 8 + 64 units of the sum of the magnitudes. In the decode step SwiGLU's
output passes that on, takes 64 units of its own and is rounded to bf16 (half a step, 2^-8); the output is rounded once."""
import numpy as np
import pytest
import torch

from oracle import train_oracle as R
from ragged_grouped_gemm_device_gb300 import _lib
from ragged_grouped_gemm_device_gb300.layer import Int4ExpertLayer
from rounding import within_one_rounding

pytestmark = pytest.mark.gpu
U = 2.0 ** -23


def _weights(matrices, N, K, group, seed=0, zeros=True):
    """(device tensors codes, scales, zeros; fp64 weights) of random codes."""
    rng = np.random.default_rng([matrices, N, K, group, seed])
    groups = (K + group - 1) // group
    codes = rng.integers(0, 16, (matrices, N, K)).astype(np.uint8)
    scales = R.to_bf16(((0.5 + rng.random((matrices, N, groups))) * K ** -0.5 / 4).astype(np.float32))
    z = rng.integers(0, 16, (matrices, N, groups)).astype(np.uint8) if zeros else None
    dev = (torch.from_numpy(R.two_to_a_byte(codes)).cuda(), torch.from_numpy(scales).bfloat16().cuda(),
           None if z is None else torch.from_numpy(z).cuda())
    return codes, dev, R.dequantize4(codes, scales, z, group)


def _pack(dev, matrices, N, K, group):
    w = torch.full((_lib.moe_workspace_bytes(_lib.OP_W4_WEIGHTS, 0, 1, matrices, K, N, group),), 0xAB, dtype=torch.uint8, device="cuda")
    _lib.moe_w4_pack(*dev, matrices, N, K, group, w)
    return w


def _x(T, K, seed=0):
    return torch.randn(T, K, generator=torch.Generator().manual_seed(T * 7919 + K + seed)).bfloat16().cuda()


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("rows,K", [(1, 1), (3, 31), (5, 77), (17, 128), (9, 1000), (300, 513)])
def test_quantize_is_exact(lib, rows, K, group):
    rng = np.random.default_rng(rows + K)
    w = R.to_bf16((rng.standard_normal((rows, K)) * np.exp(rng.standard_normal((rows, 1)))).astype(np.float32))
    w[0, : K // 2] = 0.0
    if rows > 4:
        w[3], w[4] = np.abs(w[3]), 0.0
    groups = (K + group - 1) // group
    codes = torch.full((rows, (K + 1) // 2), 0xFF, dtype=torch.uint8, device="cuda")
    scales, zeros = torch.full((rows, groups), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((rows, groups), 99, dtype=torch.uint8, device="cuda")
    _lib.moe_w4_quantize_rows(torch.from_numpy(w).bfloat16().cuda(), rows, K, group, codes, scales, zeros)
    c, s, z = R.quantize4(w, group)
    assert np.array_equal(scales.float().cpu().numpy(), s) and np.array_equal(zeros.cpu().numpy(), z)
    assert np.array_equal(codes.cpu().numpy(), R.two_to_a_byte(c))


def test_quantize_extremes(lib):
    """The largest finite values do not overflow; a NaN or an infinity makes its group's scale NaN, nothing else."""
    w = torch.zeros(2, 256, dtype=torch.bfloat16)
    top = torch.finfo(torch.bfloat16).max
    w[0, 0], w[0, 1], w[0, 130], w[1, 64], w[1, 200] = top, -top, 1e-38, float("nan"), float("-inf")
    w = w.cuda()
    codes, scales = torch.empty(2, 128, dtype=torch.uint8, device="cuda"), torch.empty(2, 4, dtype=torch.bfloat16, device="cuda")
    zeros = torch.empty(2, 4, dtype=torch.uint8, device="cuda")
    _lib.moe_w4_quantize_rows(w, 2, 256, 64, codes, scales, zeros)
    s = scales.float().cpu()
    assert torch.isfinite(s[0]).all() and s[0, 0] > 4e37 and s[1, 0] == 0 and torch.isnan(s[1, 1]) and s[1, 2] == 0 and torch.isnan(s[1, 3])


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("matrices,N,K,zeros", [(1, 1, 1, True), (2, 17, 130, True), (3, 33, 257, False), (1, 16, 128, True)])
def test_packed_layout(lib, matrices, N, K, zeros, group):
    codes, dev, _ = _weights(matrices, N, K, group, zeros=zeros)
    groups = (K + group - 1) // group
    bits = dev[1].view(torch.int16).cpu().numpy().view(np.uint16)
    z = dev[2].cpu().numpy() if zeros else np.full((matrices, N, groups), 8, np.uint8)
    want = R.pack4(codes, bits, z, group)
    got = _pack(dev, matrices, N, K, group).cpu().numpy()
    size = 1024 + 40 * (128 // group)
    pieces = matrices * ((N + 15) // 16) * ((K + 127) // 128)
    for i in range(pieces):   # what pads a piece need not be written
        at = i * ((size + 15) // 16 * 16)
        assert np.array_equal(got[at:at + size], want[at:at + size])


def _check_matvec(x, ids, k, w, y):
    xs, out = x.double().cpu().numpy(), y.double().cpu().numpy()
    n = out.shape[0]
    K = xs.shape[1]
    idh = np.zeros(n, np.int64) if ids is None else ids.cpu().numpy().reshape(-1)
    for s in range(n):
        if not 0 <= idh[s] < w.shape[0]:
            assert (out[s] == 0).all()
            continue
        ref = w[idh[s]] @ xs[s // k]
        tol = (K / 8 + 64) * U * (np.abs(w[idh[s]]) @ np.abs(xs[s // k]))
        assert within_one_rounding(out[s], ref, tol, y.dtype), (s, idh[s])


# one token to several tiles of tokens, one matrix and many, odd widths and lengths, both output types
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T,k,matrices,N,K", [(1, 1, 1, 16, 128), (1, 1, 1, 1, 1), (1, 1, 1, 300, 1000), (3, 1, 1, 64, 513), (8, 1, 1, 48, 256),
                                              (9, 1, 1, 130, 384), (40, 1, 1, 64, 200), (70, 1, 2, 33, 130), (1, 4, 7, 40, 640),
                                              (5, 3, 4, 100, 136), (33, 8, 16, 24, 128), (2, 2, 5, 17, 2100), (1, 1, 1, 2048, 8192)])
def test_matvec(lib, T, k, matrices, N, K, group):
    _, dev, w = _weights(matrices, N, K, group, zeros=(K % 2 == 0))
    packed = _pack(dev, matrices, N, K, group)
    x = _x(T, K)
    ids = None
    if matrices > 1 or k > 1:
        ids = torch.randint(-1, matrices + 1, (T, k), generator=torch.Generator().manual_seed(N), dtype=torch.int32).cuda()
    for t in (torch.bfloat16, torch.float32):
        y = torch.full((T * k, N), float("nan"), dtype=t, device="cuda")
        _lib.moe_w4_matvec(x, ids, T, k, matrices, N, K, group, packed, y)
        _check_matvec(x, ids, k, w, y)


def test_matvec_of_rows_in_wider_buffers(lib):
    T, N, K, group = 5, 70, 264, 64
    _, dev, w = _weights(1, N, K, group)
    packed = _pack(dev, 1, N, K, group)
    x = _x(T, K + 13)
    for at in (3, 8):
        out = torch.full((T, N + 9), float("nan"), device="cuda")
        _lib.moe_w4_matvec(x[:, at:at + K] if at == 3 else x[:, at:at + K], None, T, 1, 1, N, K, group, packed, out[:, 5:5 + N])
        _check_matvec(x[:, at:at + K], None, 1, w, out[:, 5:5 + N])
        assert torch.isnan(out[:, :5]).all() and torch.isnan(out[:, 5 + N:]).all()
    one = x[:1, :K].expand(T, K)                                            # one row for all tokens
    y = torch.empty(T, N, device="cuda")
    _lib.moe_w4_matvec(one, None, T, 1, 1, N, K, group, packed, y)
    assert torch.equal(y, y[:1].expand(T, N))


def _experts(E, d, h, group, seed=0):
    _, ug, wug = _weights(2 * E, h, d, group, seed)
    _, down, wd = _weights(E, d, h, group, seed + 1)
    return ug, down, wug[0::2], wug[1::2], wd


def _route(T, E, k, seed=0, invalid=True):
    g = torch.Generator().manual_seed(100 * T + E + k + seed)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32) if T else torch.empty(0, k, dtype=torch.int32)
    if invalid and T > 1:
        drop = torch.rand(T, k, generator=g) < 0.15
        ids[drop] = torch.where(torch.rand(int(drop.sum()), generator=g) < 0.5, -1, E).to(torch.int32)
        ids[T // 2] = -1                                                    # a token without experts
    return ids.cuda(), torch.rand(T, k, generator=g).cuda()


def _check_decode(x, ids, weights, gate, up, down, out):
    ref, mag, amag = R.swiglu4(x.double().cpu().numpy(), ids.cpu().numpy(), None if weights is None else weights.double().cpu().numpy(), gate, up, down)
    d, h = x.shape[1], gate.shape[1]
    tol = (d / 8 + 64) * U * amag + (2.0 ** -8 + (h / 8 + 128) * U) * mag
    assert within_one_rounding(out.double().cpu().numpy(), ref, tol, torch.bfloat16)
    # the roundings to bf16 are independent: their sum is far below its bound (a lost term is not)
    if mag.size >= 64:
        assert np.linalg.norm(out.double().cpu().numpy() - ref) <= 2.0 ** -7 * np.linalg.norm(ref) + 1e-30


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T,E,k,d,h", [(1, 8, 2, 256, 128), (1, 1, 1, 64, 16), (1, 16, 8, 513, 77), (2, 4, 3, 128, 96), (7, 6, 2, 100, 45),
                                       (16, 32, 8, 192, 64), (33, 4, 4, 136, 48), (64, 16, 8, 64, 33), (40, 1, 1, 256, 128), (20, 3, 1, 1000, 200),
                                       (3, 40, 32, 64, 32)])
def test_decode(lib, T, E, k, d, h, group):
    ug, down, gate, up, wd = _experts(E, d, h, group)
    layer = Int4ExpertLayer.from_checkpoint(ug, down, E, d, h, group)
    x = _x(T, d)
    ids, weights = _route(T, E, k)
    out = layer.forward(x, ids, weights)
    _check_decode(x, ids, weights, gate, up, wd, out)
    assert torch.equal(out, layer.forward(x, ids, weights).clone())          # a fixed order
    ones = torch.empty_like(out)
    _lib.moe_w4_swiglu_decode(x, ids, None, T, k, E, d, h, group, layer.w_ug, layer.w_down, ones, layer.ws)
    _check_decode(x, ids, None, gate, up, wd, ones)


def test_the_same_expert_twice(lib):
    """A token may name an expert twice: both slots count."""
    E, d, h, group, T, k = 3, 128, 64, 64, 9, 4
    ug, down, gate, up, wd = _experts(E, d, h, group)
    layer = Int4ExpertLayer.from_checkpoint(ug, down, E, d, h, group)
    x, ids, weights = _x(T, d), torch.randint(0, 2, (T, k), dtype=torch.int32).cuda(), torch.rand(T, k).cuda()
    ids[0] = 1
    _check_decode(x, ids, weights, gate, up, wd, layer.forward(x, ids, weights))


@pytest.mark.parametrize("E,k,d,h,group", [(40, 8, 256, 1024, 64), (24, 4, 1024, 300, 32), (64, 8, 136, 520, 128)])
def test_popular_experts_in_many_blocks(lib, E, k, d, h, group):
    """Experts with more slots than a group of eight takes, whose tiles are spread over many blocks: every block has to find the
    same slots in a group, or some are left out. Work and output buffers start as NaN."""
    ug, down, gate, up, wd = _experts(E, d, h, group)
    layer = Int4ExpertLayer.from_checkpoint(ug, down, E, d, h, group)
    T = 48
    x = _x(T, d)
    g = torch.Generator().manual_seed(E)
    ids = torch.sort(torch.randn(T, E, generator=g) + 2.0 * torch.randn(E, generator=g), dim=1, descending=True).indices[:, :k].to(torch.int32)
    assert int(torch.bincount(ids.flatten().long()).max()) > 16
    weights = torch.rand(T, k, generator=g).cuda()
    layer._buffers(T, k)
    layer.ws.fill_(255)
    layer.out.fill_(float("nan"))
    first = layer.forward(x, ids.cuda(), weights).clone()
    _check_decode(x, ids.cuda(), weights, gate, up, wd, first)
    layer.ws.fill_(255)
    assert torch.equal(first, layer.forward(x, ids.cuda(), weights))
    y = torch.full((T * k, h), float("nan"), device="cuda")
    _lib.moe_w4_matvec(x, ids.cuda(), T, k, 2 * E, h, d, group, layer.w_ug, y)
    w = np.stack([gate, up], axis=1).reshape(2 * E, h, d)
    _check_matvec(x, ids.cuda(), k, w, y)


# rows whose x goes through shared memory in several segments (one token, few and many of an expert, either product), and the
# limits of slots and experts
@pytest.mark.parametrize("T,E,k,d,h,group", [(1, 4, 2, 4400, 4300, 64), (6, 4, 2, 4400, 136, 32), (12, 3, 1, 64, 4300, 128), (30, 2, 2, 4400, 2200, 64),
                                             (25, 2, 1, 2064, 2056, 32), (128, 1024, 32, 64, 16, 32), (128, 400, 32, 40, 24, 64)])
def test_long_rows_and_limits(lib, T, E, k, d, h, group):
    ug, down, gate, up, wd = _experts(E, d, h, group)
    layer = Int4ExpertLayer.from_checkpoint(ug, down, E, d, h, group)
    x = _x(T, d)
    ids, weights = _route(T, E, k)
    layer._buffers(T, k)
    layer.ws.fill_(255)
    out = layer.forward(x, ids, weights).clone()
    _check_decode(x, ids, weights, gate, up, wd, out)
    layer.ws.fill_(255)
    assert torch.equal(out, layer.forward(x, ids, weights))
    y = torch.full((T * k, h), float("nan"), device="cuda")
    ids2 = torch.where(ids >= 0, 2 * ids + 1, ids)  # the up matrices
    _lib.moe_w4_matvec(x, ids2, T, k, 2 * E, h, d, group, layer.w_ug, y)
    w = np.stack([gate, up], axis=1).reshape(2 * E, h, d)
    _check_matvec(x, ids2, k, w, y)


def test_more_slots_than_one_call_takes(lib):
    E, d, h, group, T, k = 5, 64, 32, 32, 700, 8
    ug, down, gate, up, wd = _experts(E, d, h, group)
    layer = Int4ExpertLayer.from_checkpoint(ug, down, E, d, h, group)
    x = _x(T, d)
    ids, weights = torch.randint(0, E, (T, k), dtype=torch.int32).cuda(), torch.rand(T, k).cuda()
    out = layer.forward(x, ids, weights).clone()
    _check_decode(x, ids, weights, gate, up, wd, out)
    with pytest.raises(_lib.MoEError):
        _lib.moe_w4_swiglu_decode(x, ids, weights, T, k, E, d, h, group, layer.w_ug, layer.w_down, out, torch.empty(1 << 22, dtype=torch.uint8, device="cuda"))
    assert layer.forward(x[:0], ids[:0], weights[:0]).shape == (0, d)


def test_a_bad_token_stays_alone(lib):
    E, d, h, group, T, k = 4, 256, 64, 128, 12, 2
    ug, down, *_ = _experts(E, d, h, group)
    layer = Int4ExpertLayer.from_checkpoint(ug, down, E, d, h, group)
    x = _x(T, d)
    ids, weights = _route(T, E, k, invalid=False)
    clean = layer.forward(x, ids, weights).clone()
    x[3, 5], x[8, 200] = float("nan"), float("inf")
    got = layer.forward(x, ids, weights)
    rest = [i for i in range(T) if i not in (3, 8)]
    assert torch.isnan(got[3]).all() and torch.equal(got[rest], clean[rest]) and not torch.isfinite(got[8]).all()


def test_layer_from_bf16_weights(lib):
    """Quantized once from the weights of ExpertLayer: the values that the codes stand for are what is multiplied."""
    E, d, h, k, T = 6, 160, 96, 2, 11
    g = torch.Generator().manual_seed(2)
    w_ug = (torch.randn(E, 2 * h, d, generator=g) * d ** -0.5).bfloat16().cuda()
    w_down = (torch.randn(E, h, d, generator=g) * h ** -0.5).bfloat16().cuda()
    for group in (32, 128):
        layer = Int4ExpertLayer(w_ug, w_down, group)
        deq = lambda w: R.dequantize4(*R.quantize4(w.float().cpu().numpy().reshape(-1, w.shape[-1]), group), group).reshape(w.shape)
        wug, wd = deq(w_ug), deq(w_down.transpose(1, 2).contiguous())
        x = _x(T, d)
        ids, weights = _route(T, E, k)
        _check_decode(x, ids, weights, wug[:, :h], wug[:, h:], wd, layer.forward(x, ids, weights))


def test_streams_and_graphs(lib):
    E, d, h, group, T, k = 8, 256, 128, 64, 5, 3
    ug, down, *_ = _experts(E, d, h, group)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    layer, other = (Int4ExpertLayer.from_checkpoint(ug, down, E, d, h, group, stream=s) for s in (None, side))
    x = _x(T, d)
    ids, weights = _route(T, E, k)
    want = layer.forward(x, ids, weights).clone()
    side.wait_stream(torch.cuda.current_stream())
    got = other.forward(x, ids, weights, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer.forward(x, ids, weights)
    x.mul_(-0.5)
    ids.copy_(_route(T, E, k, seed=9)[0])
    graph.replay()
    got = got.clone()
    assert torch.equal(got, layer.forward(x, ids, weights))


def test_refusals(lib):
    E, d, h, group, T, k = 4, 64, 32, 32, 3, 2
    ug, down, *_ = _experts(E, d, h, group)
    layer = Int4ExpertLayer.from_checkpoint(ug, down, E, d, h, group)
    x = _x(T, d)
    ids, weights = _route(T, E, k)
    for bad in ((x.float(), ids, weights), (x[:, :32], ids, weights), (x, ids.long(), weights), (x, ids, weights.double()), (x, ids[:2], weights)):
        with pytest.raises(ValueError):
            layer.forward(*bad)
    out, ws = torch.empty_like(x), torch.empty(1 << 16, dtype=torch.uint8, device="cuda")
    call = lambda **a: _lib.moe_w4_swiglu_decode(**{**dict(x=x, ids=ids, weights=weights, T=T, top_k=k, E=E, d=d, h=h, group=group, w_ug=layer.w_ug,
                                                          w_down=layer.w_down, out=out, ws=ws), **a})
    call()
    for bad in (dict(w_ug=layer.w_ug[:-1]), dict(w_down=layer.w_down[:-1]), dict(ids=ids[:1]), dict(x=x.cpu()), dict(out=out.float())):
        with pytest.raises(ValueError):
            call(**bad)
    for bad in (dict(ws=None), dict(group=48), dict(w_ug=torch.empty(layer.w_ug.numel() + 16, dtype=torch.uint8, device="cuda")[16:])):
        with pytest.raises(_lib.MoEError):
            call(**bad)
