"""AdamW over many tensors against the fp64 reference.

Tolerances. m, v and the update are a handful of fp32 roundings (unit 2^-24) of their terms; the bias corrections take
expm1 of a product, 8 units more. A bf16 parameter is rounded up or down by the given random bits: exactly as the reference
where the fraction and u are further from the threshold than the fp32 error is. The same holds for 8-bit states: elements have
4 significant bits, so an error of 16 units is 16 * 2^-24 * 2^4 = 2^-16 of a step."""
import math

import numpy as np
import pytest
import torch

from oracle import train_oracle as R
from ragged_grouped_gemm_device_gb300 import _lib
from ragged_grouped_gemm_device_gb300.optim import AdamW

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
SIZES = [1, 31, 32, 33, 4095, 4096, 4097, 100000, 0, 7, 12345]


def _make(sizes, p_dtype, g_dtype, seed=0, offset=0):
    """Tensors of the sizes, each `offset` elements off an allocation's alignment."""
    g = torch.Generator().manual_seed(seed)
    n = lambda size, std, t: (torch.randn(size + offset, generator=g) * std).to(t).cuda()[offset:]
    return [n(s, 0.05, p_dtype) for s in sizes], [n(s, 1e-3, g_dtype) * (1 + i % 3) for i, s in enumerate(sizes)]


def _load8(code, scale, n):
    v = code[:n].view(torch.float8_e4m3fn).double().cpu().numpy()
    s = scale.cpu().numpy().astype(np.int64) - 127
    return v * np.repeat(np.ldexp(1.0, s), 32)[:n]


def _host(t):
    return t.detach().double().cpu().numpy()


def _check_step(opt, grads, sizes, before, c=1.0, lr=None):
    """Against the reference from the state `before` the step: lists of p, m, v (fp64) and the step's number."""
    t = before["t"]
    lr = opt.lr if lr is None else lr
    for j, n in enumerate(sizes):
        if n == 0:
            continue
        at = opt.starts[j]
        decay = opt._table[j].weight_decay
        p, m, v = R.adamw(before["p"][j], _host(grads[j]), before["m"][j], before["v"][j], t, lr, *opt.betas, opt.eps, decay, c)
        g = c * _host(grads[j])
        em = 8 * U * (np.abs(opt.betas[0] * before["m"][j]) + np.abs((1 - opt.betas[0]) * g))
        ev = 8 * U * v
        # the update's error: em's share, and 32 units of it (root, quotient, bias corrections, rate)
        denominator = np.sqrt(v / (1 - opt.betas[1] ** t)) + opt.eps
        ep = 2 * U * np.abs(before["p"][j]) + 2 * U * np.abs(p) + lr / (1 - opt.betas[0] ** t) * (em + 32 * U * np.abs(m)) / denominator
        got = _host(opt.params[j])
        bits = R.random_bits(opt.seed, t, j, n).astype(np.int64)
        if opt.params[j].dtype == torch.bfloat16:
            want, step, far = R.round_up_where(np.abs(p), ((bits >> 8) & 0xFFFF) / 65536, 7, -126)
            sure = far > ep / step
            assert (got[sure] == (np.sign(p) * want)[sure]).all()
            assert sure.mean() > 0.9 and (np.abs(got - p) <= step + ep).all()
        else:
            assert (np.abs(got - p) <= ep).all()
            if opt.copies[j] is not None:
                assert torch.equal(opt.copies[j], opt.params[j].bfloat16())
        if opt.state_bits == 32:
            assert (np.abs(_host(opt.m[at:at + n]) - m) <= em).all() and (np.abs(_host(opt.v[at:at + n]) - v) <= ev).all()
            continue
        blocks = (n + 31) // 32
        for name, x, u, keep in (("m", m, bits & 0xFFFF, False), ("v", np.sqrt(v), bits >> 16, True)):
            code, scale = getattr(opt, name)[at:at + n], getattr(opt, name + "_scale")[at // 32:at // 32 + blocks]
            want, s, far = R.quantize8(x, u / 65536, keep)
            top = np.abs(R._blocks(x)).max(axis=1) / np.ldexp(448.0, s)
            edge = (np.abs(top - 1) < 2e-6) | (np.abs(top - 0.5) < 2e-6)     # the block's scale may go either way
            assert ((scale.cpu().numpy().astype(np.int64) - 127 == s) | edge).all()
            em8 = np.divide(em, np.abs(m), out=np.zeros_like(m), where=m != 0) if name == "m" else 8 * U
            sure = (far > 2.0 ** -16 + 16 * em8) & ~np.repeat(edge, 32)[:n]
            if keep:
                sure |= (want == 2.0 ** -9) & ~np.repeat(edge, 32)[:n]
            got = code.view(torch.float8_e4m3fn).double().cpu().numpy()
            assert (got[sure] == want[sure]).all()
            # how many are sure: the largest bf16 gradient of a block has one of 128 mantissas, and one of them may put the block
            # at the border, so of 129 blocks one is expected there; more than 12 (Poisson) has a probability below 1e-9. The
            # thresholds' own share is 2 * (2^-16 + 16 * 2^-20)
            assert n < 4095 or sure.mean() > 0.9


def _state(opt, sizes, t):
    one = lambda j, n, name: (_host(getattr(opt, name)[opt.starts[j]:opt.starts[j] + n]) if opt.state_bits == 32 else
                              _load8(getattr(opt, name)[opt.starts[j]:], getattr(opt, name + "_scale")[opt.starts[j] // 32:
                                     opt.starts[j] // 32 + (n + 31) // 32], n))
    v = [one(j, n, "v") for j, n in enumerate(sizes)]
    return {"t": t, "p": [_host(p) for p in opt.params], "m": [one(j, n, "m") for j, n in enumerate(sizes)],
            "v": [x * x for x in v] if opt.state_bits == 8 else v}


@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("g_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("p", ["fp32", "copy", "bf16"])
@pytest.mark.parametrize("bits", [32, 8])
def test_steps_match_the_reference(lib, bits, p, g_dtype, offset):
    params, grads = _make(SIZES, torch.bfloat16 if p == "bf16" else torch.float32, g_dtype, offset=offset)
    copies = None
    if p == "copy":
        copies = [torch.zeros(n + offset, dtype=torch.bfloat16, device="cuda")[offset:] for n in SIZES]
    opt = AdamW(params, lr=2e-3, betas=(0.9, 0.95), eps=1e-8, weight_decay=[0.1 * (i % 2) for i in range(len(SIZES))], state_bits=bits,
                copies=copies, seed=77)
    for t in range(1, 4):
        before = _state(opt, SIZES, t)
        opt.step(grads)
        assert opt.steps == t and int(opt._steps[1]) == 0
        _check_step(opt, grads, SIZES, before)
        grads = [g * 0.7 for g in grads]
    # the room between two parameters stays 0
    live = torch.zeros(opt.m.numel(), dtype=torch.bool)
    for at, n in zip(opt.starts, SIZES):
        live[at:at + n] = True
    assert (opt.m.cpu()[~live] == 0).all() and (opt.v.cpu()[~live] == 0).all()


@pytest.mark.parametrize("size", [1e18, 1e-12])
@pytest.mark.parametrize("bits", [32, 8])
def test_states_of_any_size(lib, bits, size):
    """Gradients of about 1e15, whose 8-bit scales are above 2^38, and of 1e-15."""
    sizes = [100, 4500]
    params, grads = _make(sizes, torch.float32, torch.float32, seed=4)
    grads = [g * size for g in grads]
    opt = AdamW(params, lr=1e-3, state_bits=bits, seed=5)
    for t in (1, 2):
        before = _state(opt, sizes, t)
        opt.step(grads)
        _check_step(opt, grads, sizes, before)


def test_no_gradient_and_the_smallest_eps(lib):
    """0 / eps is 0 for every eps above 0."""
    for bits in (32, 8):
        for eps in (1e-8, 1e-37, 1e-40, 1e-300):
            p = torch.ones(70, device="cuda")
            opt = AdamW([p], eps=eps, weight_decay=0.0, state_bits=bits)
            opt.step([torch.zeros_like(p)])
            assert (p == 1.0).all()


def test_more_tensors_than_one_launch_takes(lib):
    sizes = [1 + (i * 37) % 300 for i in range(300)]
    for bits in (32, 8):
        params, grads = _make(sizes, torch.float32, torch.float32)
        opt = AdamW(params, lr=1e-3, weight_decay=0.1, state_bits=bits, max_norm=1e-2)
        before = _state(opt, sizes, 1)
        norm = float(opt.step(grads))
        want = math.sqrt(sum(float((_host(g) ** 2).sum()) for g in grads))
        assert abs(norm - want) <= 32 * U * want
        _check_step(opt, grads, sizes, before, c=float(opt._norm[1]))
        assert opt.steps == 1


@pytest.mark.parametrize("g_dtype", [torch.float32, torch.bfloat16])
def test_norm_and_clipping(lib, g_dtype):
    sizes = [5, 4096, 1000003, 0, 12]
    params, grads = _make(sizes, torch.float32, g_dtype)
    want = math.sqrt(sum(float((_host(g) ** 2).sum()) for g in grads))
    # pieces of 4096: 16 squares a thread and a tree of 8 levels in fp32, the rest in fp64; a root halves
    tol = 16 * U * want
    for max_norm in (want * 2, want / 3):
        opt = AdamW(params, max_norm=max_norm)
        before = _state(opt, sizes, 1)
        norm = float(opt.step(grads))
        c = float(opt._norm[1])
        assert abs(norm - want) <= tol and abs(c - min(1.0, max_norm / want)) <= 20 * U
        _check_step(opt, grads, sizes, before, c=c)
    assert float(opt.step([torch.zeros_like(g) for g in grads])) == 0.0 and float(opt._norm[1]) == 1.0
    a, b = AdamW(params, max_norm=1.0), AdamW(params, max_norm=1.0)
    assert float(a.step(grads)) == float(b.step(grads))                    # a fixed order


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_norm_that_is_not_finite_skips_the_step(lib, bad):
    for bits in (32, 8):
        params, grads = _make([100, 5000], torch.float32, torch.float32)
        opt = AdamW(params, state_bits=bits, max_norm=1.0)
        opt.step(grads)
        keep = [t.clone() for t in (*params, opt.m, opt.v)]
        grads[1][4321] = bad
        norm = float(opt.step(grads))
        assert not math.isfinite(norm) and opt.steps == 1
        assert all(torch.equal(a, b) for a, b in zip(keep, (*params, opt.m, opt.v)))


def test_nan_without_clipping_stays_where_it_is(lib):
    """fp32 states: in its element. 8 bits: in its block of 32 (scale 0xFF); the rest as without it."""
    for bits in (32, 8):
        runs = []
        for bad in (False, True):
            params, grads = _make([400], torch.float32, torch.float32)
            if bad:
                grads[0][100] = float("nan")
            opt = AdamW(params, state_bits=bits)
            opt.step(grads)
            opt.step(_make([400], torch.float32, torch.float32)[1])
            runs.append(params[0].clone())
        nan = torch.isnan(runs[1]).cpu()
        where = torch.zeros(400, dtype=torch.bool)
        if bits == 32:
            where[100] = True
        else:
            where[96:128] = True
            assert opt.m_scale[3] == 255 and opt.v_scale[3] == 255
        assert torch.equal(nan, where) and torch.equal(runs[0].cpu()[~where], runs[1].cpu()[~where])


def test_8_bit_states_follow_32_bits(lib):
    """The stochastic rounding loses no small change: after many steps with a small change each, the state is where the fp32 one
    is. v moves by 0.1% of its distance a step, a sixtieth of a step of its elements. With n elements alike the mean's error is the
    single error (at most a step, 12.5%) over sqrt(n), five deviations. m has no bias. v is the square of what is rounded, so it
    gains the rounding's variance: of a change dr between two elements a step s <= r / 8 apart, dr (s - dr) < dr r / 8. On the way
    from 0 to R that is at most R^2 / 16 (the way back from the largest r, 0.5% further, adds less than a hundredth of it), or
    R / 32 of the root."""
    n = 1 << 16
    g1, g2 = torch.full((n,), 1e-3, device="cuda"), torch.full((n,), 3e-4, device="cuda")
    states = []
    for bits in (32, 8):
        p = torch.zeros(n, device="cuda")
        opt = AdamW([p], lr=1e-3, betas=(0.9, 0.999), state_bits=bits)
        for i in range(200):
            opt.step([g1 if i < 100 else g2])
        states.append((_state(opt, [n], 0), p))
    for name in ("m", "v"):
        a, b = states[0][0][name][0], states[1][0][name][0]
        if name == "v":
            a, b = np.sqrt(a), np.sqrt(b)
        off, noise = b.mean() / a.mean() - 1, 5 * 0.125 / math.sqrt(n)
        assert -noise < off < noise + (1 / 30 if name == "v" else 0.0)


def test_small_steps_of_bf16_weights_are_not_lost(lib):
    n = 1 << 16
    p = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    opt = AdamW([p], lr=1e-4, weight_decay=0.0)
    for _ in range(20):
        opt.step([torch.ones(n, device="cuda")])
    # 20 steps of 1e-4 (a bf16 step below 1 is 2^-8): the mean moves by them; its deviation is at most a step over sqrt(n)
    assert abs(float(p.double().mean()) - (1 - 20e-4)) < 5 * 2.0 ** -8 / math.sqrt(n)


def test_graph_streams_and_learning_rate_on_the_device(lib):
    params, grads = _make([1000, 70], torch.float32, torch.float32)
    ref = [p.clone() for p in params]
    scale = torch.ones(1, device="cuda")
    a, b = AdamW(params, state_bits=8, max_norm=1e-3, lr_scale=scale), AdamW(ref, state_bits=8, max_norm=1e-3)
    a.step(grads)
    b.step(grads)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.step(grads)
    for i in range(3):
        scale.fill_(0.5 ** i)
        graph.replay()
        b.lr = 1e-3 * 0.5 ** i
        b.step(grads)
    assert a.steps == b.steps == 4 and all(torch.equal(p, q) for p, q in zip(params, ref))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a.step(grads, stream=side)
    side.synchronize()
    b.lr = 1e-3 * 0.25
    b.step(grads)
    assert all(torch.equal(p, q) for p, q in zip(params, ref))


def test_checkpoint_goes_on_and_versions_count(lib):
    params, grads = _make([777, 64], torch.float32, torch.float32)
    opt = AdamW(params, state_bits=8, seed=5)
    opt.step(grads)
    p2 = [p.clone() for p in params]
    two = AdamW(p2, state_bits=8, seed=5)
    for n in ("m", "v", "m_scale", "v_scale"):
        getattr(two, n).copy_(getattr(opt, n))
    two.steps = opt.steps
    version = params[0]._version
    opt.step(grads)
    two.step(grads)
    assert all(torch.equal(p, q) for p, q in zip(params, p2)) and params[0]._version > version


def test_refusals(lib):
    p, g = torch.zeros(10, device="cuda"), torch.zeros(10, device="cuda")
    for bad in (dict(params=[]), dict(params=[p.half()]), dict(params=[p.cpu()]), dict(params=[torch.zeros(4, 4, device="cuda").t()[1:]]),
                dict(params=[p], state_bits=16), dict(params=[p], weight_decay=[0.1, 0.2]), dict(params=[p], copies=[g]),
                dict(params=[p.bfloat16()], copies=[p.bfloat16()]), dict(params=[p], max_norm=0.0),
                dict(params=[p, g, p]), dict(params=[p[:6], p[5:]]), dict(params=[p], copies=[p.view(torch.bfloat16)[:10]])):
        with pytest.raises(ValueError):
            AdamW(**bad)
    opt = AdamW([p])
    for bad in ([], [g, g], [g[:5]], [g.double()], [g.cpu()]):
        with pytest.raises(ValueError):
            opt.step(bad)
    with pytest.raises(_lib.MoEError):
        AdamW([p], betas=(1.0, 0.9)).step([g])
    with pytest.raises(_lib.MoEError):
        AdamW([p], lr=float("nan")).step([g])
    AdamW([p[:5], p[5:], p[5:5]]).step([g[:5], g[5:], g[5:5]])
