"""The router's gate against the fp64 reference: ids and counts exactly, floats to the rounding of their
terms. An exponential of x is off by at most 2 + 1.5 |x| units of 2^-23 (its argument is rounded
once after scaling), a sum by one unit a level; `rtol` below covers a row's largest |logit - max|."""
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


class Gate:
    def __init__(self, logits, mask, k, renorm, seed=0):
        T, E = logits.shape
        nan = lambda *s, dtype=torch.float32: torch.full(s, float("nan"), dtype=dtype, device="cuda")
        junk = lambda *s: torch.full(s, -77, dtype=torch.int32, device="cuda")
        self.T, self.E, self.k, self.flags = T, E, k, _lib.GATE_RENORM if renorm else 0
        self.logits, self.mask, self.renorm = logits, mask, renorm
        self.ids, self.weights, self.lse = junk(T, k), nan(T, k), nan(T)
        self.counts, self.n, self.prob_sum, self.loss = junk(E), junk(1), nan(E), nan(2)
        self.dlogits = torch.full_like(logits, float("nan"), memory_format=torch.contiguous_format)
        self.ws = torch.full((max(1, _lib.moe_workspace_bytes(_lib.OP_GATE, T, k, E)),), 0xA5, dtype=torch.uint8, device="cuda")
        g = torch.Generator().manual_seed(seed)
        self.d_weights = torch.randn(T, k, generator=g).cuda()
        self.d_loss = torch.tensor([0.6 * max(T, 1), -0.2 * max(T, 1)], device="cuda")

    def run(self):
        _lib.moe_gate_fwd(self.logits, self.mask, self.T, self.k, self.E, self.flags, self.ids, self.weights, self.lse,
                          self.counts, self.n, self.prob_sum, self.loss, self.ws)
        _lib.moe_gate_bwd(self.logits, self.lse, self.ids, self.weights, self.counts, self.n, self.d_weights, self.d_loss,
                          self.T, self.k, self.E, self.flags, self.dlogits)
        torch.cuda.synchronize()
        return self

    def check(self):
        lg = _host(self.logits)
        mask = None if self.mask is None else self.mask.bool().cpu().numpy()
        r = B.gate(lg, mask, self.k, self.renorm)
        assert np.array_equal(self.ids.cpu().numpy(), r["ids"])
        assert np.array_equal(self.counts.cpu().numpy(), r["counts"]) and int(self.n) == r["n"]
        finite = np.where(np.isfinite(lg), lg, 0.0)
        reach = np.abs(finite).max() * 2 if lg.size else 0.0
        rtol = U32 * (32 + 6 * reach)
        assert (np.abs(_host(self.weights) - r["weights"]) <= rtol * r["weights"]).all()
        on = r["lse"] != -np.inf
        lse = _host(self.lse)
        assert np.array_equal(lse == -np.inf, ~on)
        assert (np.abs(lse[on] - r["lse"][on]) <= rtol * (1 + np.abs(r["lse"][on]))).all()
        depth = self.T / 4864 + 64
        assert (np.abs(_host(self.prob_sum) - r["prob_sum"]) <= (rtol + depth * U32) * r["prob_sum"]).all()
        # lse^2 doubles lse's relative error, which is absolute where lse is near 0
        slack = np.array([2 * (rtol + depth * U32), 0.0]) * r["loss"]
        if on.any():
            slack[1] = 2 * (rtol + depth * U32) * ((1 + np.abs(r["lse"][on])) ** 2).mean()
        assert (np.abs(_host(self.loss) - r["loss"]) <= slack).all()
        want, mag = B.gate_grad(r, self.k, self.renorm, _host(self.d_weights), _host(self.d_loss))
        assert within_one_rounding(_host(self.dlogits), want, 4 * rtol * mag, self.logits.dtype)


def _logits(T, E, dtype, seed=0):
    g = torch.Generator().manual_seed(7 * T + E + seed)
    return (torch.randn(T, E, generator=g) + 0.5 * torch.randn(E, generator=g)).to(TYPES[dtype]).cuda()


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 4, 2), (16, 128, 8), (3, 8, 8), (5, 33, 3), (9, 32, 32), (65, 60, 6),
                                   (40, 64, 1), (33, 129, 8), (20, 256, 8), (11, 257, 7), (8, 512, 4), (7, 1000, 10),
                                   (5, 1024, 32), (5000, 16, 2)])
def test_matches_the_reference(lib, T, E, k, dtype, renorm):
    Gate(_logits(T, E, dtype), None, k, renorm).run().check()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("E,k", [(128, 8), (200, 9), (512, 4), (1000, 3), (100, 5)])
def test_many_tokens_at_every_width(lib, E, k, dtype):
    """Enough tokens for the narrow lane groups of the forward (E = 100: rows that are read one element at
    a time stay at full width)."""
    Gate(_logits(5000, E, dtype), None, k, E % 200 == 0).run().check()


@pytest.mark.parametrize("renorm", [True, False])
def test_masked_tokens_and_excluded_experts(lib, renorm):
    """Padding tokens, experts at -inf (fewer than k left in some rows, none in one), the type's lowest
    value, ties everywhere, and -0 next to 0."""
    T, E, k = 70, 40, 6
    lg = _logits(T, E, "fp32")
    lg[3, 4:] = float("-inf")
    lg[5] = float("-inf")
    lg[8, 1::2] = torch.finfo(torch.float32).min
    lg[9] = 1.25
    lg[10] = 0.0
    lg[10, ::2] = -0.0
    lg[11] = torch.finfo(torch.float32).min
    mask = torch.ones(T, dtype=torch.bool, device="cuda")
    mask[[0, 9, 33, 69]] = False
    ok = Gate(lg, mask, k, renorm).run()
    # differences between a row's logits of 3e38 leave no accuracy bound: those rows by themselves
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[[8, 11]] = False
    assert (ok.ids[3].tolist()[4:] == [-1, -1]) and (ok.weights[3, 4:] == 0).all()
    assert (ok.ids[5] == -1).all() and (ok.weights[5] == 0).all() and (ok.dlogits[5] == 0).all()
    assert ok.ids[10].tolist() == list(range(k)) and ok.ids[11].tolist() == list(range(k))
    assert torch.allclose(ok.weights[11], torch.full((k,), 1 / k if renorm else 1 / E, device="cuda"))
    assert set(ok.ids[8].tolist()) <= set(range(0, E, 2)) and torch.isfinite(ok.dlogits[keep]).all()
    lg[8], lg[11] = lg[1], lg[2]
    Gate(lg, mask, k, renorm).run().check()
    Gate(lg, torch.zeros(T, dtype=torch.uint8, device="cuda"), k, renorm).run().check()  # nobody takes part


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_nan_and_infinity(lib, value):
    """A NaN is never selected; it and +inf make their token's weights NaN and leave other tokens'."""
    lg = _logits(12, 24, "bf16")
    clean = Gate(lg.clone(), None, 4, True).run()
    lg[5, 3] = value
    got = Gate(lg, None, 4, True).run()
    others = [t for t in range(12) if t != 5]
    assert torch.equal(got.ids[others], clean.ids[others]) and torch.equal(got.weights[others], clean.weights[others])
    assert torch.isnan(got.weights[5]).all() and torch.isnan(got.dlogits[5]).all() and torch.isnan(got.loss).all()
    assert ((got.ids[5] >= 0) & (got.ids[5] < 24)).all()
    if value != value:
        assert 3 not in got.ids[5].tolist()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_strided_logits_and_parts_of_the_gradient(lib, dtype):
    T, E, k = 50, 48, 4
    wide = _logits(T, 3 * E + 5, dtype)
    lg = wide[:, E + 1:2 * E + 1]
    Gate(lg, None, k, True).run().check()
    one = wide[:1, :E].expand(T, E)
    Gate(one, None, k, False).run().check()
    # without one of the upstream gradients: what zeros in its place give, to the last bit
    g = Gate(lg.contiguous(), None, k, False).run()
    for which in ("d_weights", "d_loss"):
        keep = getattr(g, which)
        setattr(g, which, torch.zeros_like(keep))
        want = g.run().dlogits.clone()
        setattr(g, which, None)
        assert torch.equal(g.run().dlogits, want)
        setattr(g, which, keep)
    # ids and weights alone are those of the full call
    ids, w = torch.empty_like(g.ids), torch.empty_like(g.weights)
    _lib.moe_gate_fwd(g.logits, None, T, k, E, 0, ids, w)
    assert torch.equal(ids, g.ids) and torch.equal(w, g.weights)


def test_many_tokens_repeat_bit_for_bit_and_route(lib):
    """More tokens than one pass of the grid; every sum in a fixed order; the ids and counts agree
    with moe_route_offsets, which drops the padding tokens' slots."""
    T, E, k = 20000, 96, 5
    mask = torch.rand(T, generator=torch.Generator().manual_seed(3)).cuda() > 0.2
    g = Gate(_logits(T, E, "bf16"), mask, k, False).run()
    first = [t.clone() for t in (g.ids, g.weights, g.prob_sum, g.loss, g.dlogits)]
    g.run().check()
    assert all(torch.equal(a, b) for a, b in zip(first, (g.ids, g.weights, g.prob_sum, g.loss, g.dlogits)))
    i32 = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")
    counts, offsets, src, inv = i32(E), i32(E), i32(T * k), i32(T * k)
    ws = torch.empty(_lib.moe_workspace_bytes(_lib.OP_ROUTE, T, k, E), dtype=torch.uint8, device="cuda")
    _lib.moe_route_offsets(g.ids, T, k, E, counts, offsets, src, inv, ws)
    assert torch.equal(counts, g.counts) and int(offsets[-1]) == int(mask.sum()) * k


def test_a_nan_loss_gradient_leaves_masked_tokens_alone(lib):
    mask = torch.tensor([True, False, True, False], device="cuda")
    g = Gate(_logits(4, 16, "bf16"), mask, 2, False)
    g.d_loss[0] = float("nan")
    g.run()
    assert torch.isnan(g.dlogits[mask]).all() and (g.dlogits[~mask] == 0).all()


def test_no_tokens(lib):
    g = Gate(torch.empty(0, 8, device="cuda"), None, 2, True).run()
    assert (g.counts == 0).all() and int(g.n) == 0 and (g.prob_sum == 0).all() and (g.loss == 0).all()


def test_refusals(lib):
    lg = _logits(4, 8, "fp32")
    g = Gate(lg, None, 2, True)
    with pytest.raises(ValueError):
        _lib.moe_gate_fwd(lg.half(), None, 4, 2, 8, 0, g.ids, g.weights)
    with pytest.raises(ValueError):
        _lib.moe_gate_fwd(lg, None, 4, 2, 8, 0, g.ids.long(), g.weights)
    with pytest.raises(ValueError):
        _lib.moe_gate_fwd(lg.t(), None, 8, 2, 4, 0, g.ids, g.weights)
    for bad in (lambda: _lib.moe_gate_fwd(lg, None, 4, 2, 8, 2, g.ids, g.weights),             # unknown flag
                lambda: _lib.moe_gate_fwd(lg, None, 4, 2, 8, 0, g.ids, g.weights, counts=g.counts),
                lambda: _lib.moe_gate_fwd(lg, None, 4, 2, 8, 0, g.ids, g.weights, None, g.counts, g.n, g.prob_sum, g.loss)):
        with pytest.raises(_lib.MoEError):
            bad()
