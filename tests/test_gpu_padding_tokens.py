"""What a block with a norm behind it and scales makes of padding tokens: the experts' rows are zeros, the join is the formula's.
Bounds: out is a handful of fp32 roundings (2^-24 each) rounded once to bf16; the gradients are sums of T terms."""
import pytest
import torch

from ragged_grouped_gemm_device_gb300.block import MoEBlock, MoEStack
from ragged_grouped_gemm_device_gb300.layer import ExpertLayer
from rounding import within_one_rounding

pytestmark = pytest.mark.gpu
T, E, k, d, h, RES, BRANCH = 40, 6, 2, 64, 40, 0.75, 0.5


def _block(post, seed=1):
    g = torch.Generator("cuda").manual_seed(seed)
    n = lambda *s, dtype=torch.float32: torch.randn(*s, generator=g, device="cuda").to(dtype)
    experts = ExpertLayer(n(E, 2 * h, d, dtype=torch.bfloat16) / 8, n(E, h, d, dtype=torch.bfloat16) / 6)
    w = dict(post_gamma=1 + 0.2 * n(d), post_beta=0.3 * n(d) if post == "layer" else None, gate=0.5 + 0.2 * n(d))
    return MoEBlock(1 + 0.2 * n(d), None, n(E, d) / 8, experts, k, pre="rms", post=post, res_scale=RES, branch_scale=BRANCH, **w)


def _inputs():
    g = torch.Generator("cuda").manual_seed(2)
    x, dout = (torch.randn(T, d, generator=g, device="cuda").bfloat16() for _ in range(2))
    return x, dout, torch.rand(T, generator=g, device="cuda") > 0.3


def _host(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("post", ["layer", "rms"])
def test_rows_and_gradients(lib, post):
    block = _block(post)
    x, dout, mask = _inputs()
    pad = ~mask
    out = block.forward(x, mask)
    beta = torch.zeros(d, device="cuda") if block.post_beta is None else block.post_beta
    z = BRANCH * block.gate.double() * beta.double()
    want = RES * x[pad].double() + z
    scale = RES * x[pad].double().abs() + z.abs()
    assert within_one_rounding(_host(out[pad]), _host(want), 8 * 2.0 ** -24 * _host(scale), torch.bfloat16)
    # only padding rows have a gradient: theirs passes to x alone, and to what makes post(0)
    only = torch.where(pad[:, None], dout, torch.zeros_like(dout))
    got = {n: t.clone() for n, t in block.backward(only).items()}
    D = only.double()
    assert within_one_rounding(_host(got["dx"]), RES * _host(D), 8 * 2.0 ** -24 * RES * _host(D.abs()), torch.bfloat16)
    for n in ("gamma", "w_router", "w_ug", "w_down", "post_gamma"):
        assert (got[n] == 0).all(), n
    near = lambda a, want, size: bool(((a.double() - want).abs() <= T * 2.0 ** -24 * size + 1e-30).all())
    assert near(got["gate"], BRANCH * beta.double() * D.sum(0), (BRANCH * beta.double() * D).abs().sum(0))
    if post == "layer":
        assert near(got["post_beta"], BRANCH * block.gate.double() * D.sum(0), (BRANCH * block.gate.double() * D).abs().sum(0))


@pytest.mark.parametrize("model", ["block", "stack"])
def test_no_share_where_the_gradient_is_zero(lib, model):
    """With dout 0 in the padding rows, what they hold changes no gradient of a weight."""
    x, dout, mask = _inputs()
    dout = torch.where(mask[:, None], dout, torch.zeros_like(dout))
    results = []
    for fill in (None, 3.0):
        blocks = [_block("layer"), _block("rms", 5)][:1 if model == "block" else 2]
        m = blocks[0] if model == "block" else MoEStack(blocks)
        m.forward(x if fill is None else torch.where(mask[:, None], x, torch.full_like(x, fill)), mask)
        got = m.backward(dout)
        assert (got["dx"][~mask] == 0).all()
        results.append([t.clone() for g in ([got] if model == "block" else got["blocks"]) for n, t in sorted(g.items()) if n != "dx"])
    assert all(torch.equal(a, b) for a, b in zip(*results))
