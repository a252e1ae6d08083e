"""What a block's or a stack's backward needs of the run before it: the same weights, whole buffers."""
import pytest
import torch

from ragged_grouped_gemm_device_gb300.block import MoEBlock, MoEStack
from ragged_grouped_gemm_device_gb300.layer import ExpertLayer
from ragged_grouped_gemm_device_gb300.optim import AdamW

pytestmark = pytest.mark.gpu

T, E, k, d, h = 24, 6, 2, 64, 40


def _block(kind, seed=1):
    g = torch.Generator("cuda").manual_seed(seed)
    n = lambda *s, dtype=torch.float32: torch.randn(*s, generator=g, device="cuda").to(dtype)
    experts = ExpertLayer(n(E, 2 * h, d, dtype=torch.bfloat16) / 8, n(E, h, d, dtype=torch.bfloat16) / 6)
    gamma, w_router = 1 + 0.2 * n(d), n(E, d) / 8
    if kind == "plain":
        return MoEBlock(gamma, 0.1 * n(d), w_router, experts, k)
    return MoEBlock(gamma, None, w_router, experts, k, pre="rms", post="layer", post_gamma=1 + 0.2 * n(d), post_beta=0.3 * n(d),
                    gate=0.5 + 0.2 * n(d), res_scale=0.75, branch_scale=0.5)


def _rows(seed=2, rows=T):
    return torch.randn(rows, d, generator=torch.Generator("cuda").manual_seed(seed), device="cuda").bfloat16()


def _model(kind):
    """(what has forward() and backward(), its blocks)"""
    if kind == "stack":
        blocks = [_block("plain"), _block("norms", 3)]
        return MoEStack(blocks), blocks
    block = _block(kind)
    return block, [block]


@pytest.mark.parametrize("kind", ["plain", "norms", "stack"])
def test_experts_changed_before_the_backward(lib, kind):
    """The backward multiplies by the experts' weights again: those of another step with this one's activations would give
    gradients of no function."""
    model, blocks = _model(kind)
    x, dout = _rows(), _rows(5)
    for b in blocks:
        for w in (b.experts.w_ug, b.experts.w_down):
            model.forward(x)
            w.mul_(1.5)
            with pytest.raises(RuntimeError, match="in place"):
                model.backward(dout)
            model.forward(x)
            model.backward(dout)
    model.forward(x)
    AdamW([blocks[-1].experts.w_down]).step([torch.ones_like(blocks[-1].experts.w_down)])
    with pytest.raises(RuntimeError, match="in place"):
        model.backward(dout)


@pytest.mark.parametrize("kind", ["plain", "norms", "stack"])
def test_a_forward_that_raises_leaves_no_run(lib, kind):
    """A mask of a wrong type is found behind the first norm, whose rows and statistics are another run's then."""
    model, _ = _model(kind)
    x, dout = _rows(), _rows(5)
    model.forward(x)
    with pytest.raises(ValueError):
        model.forward(_rows(6), torch.ones(T, device="cuda"))
    with pytest.raises(RuntimeError, match="forward"):
        model.backward(dout)
    model.forward(x)
    model.backward(dout)


@pytest.mark.parametrize("kind", ["norms", "stack"])
def test_an_output_goes_in_again(lib, kind):
    """A stack's output, whole or one row of it for all tokens, is the next input: forward and backward are
    those of a copy of it."""
    dout = _rows(5)
    for take in (lambda r: r, lambda r: r[3:4].expand(T, d)):
        results = []
        for copy in (False, True):
            model, _ = _model(kind)
            x = take(model.forward(_rows()))
            x = x.clone() if copy else x
            out = model.forward(x).clone()
            got = model.backward(dout)
            blocks = got["blocks"] if kind == "stack" else [{n: t for n, t in got.items() if n != "dx"}]
            results.append([out, got["dx"].clone()] + [b[n].clone() for b in blocks for n in sorted(b)])
        assert all(torch.equal(a, b) for a, b in zip(*results))


@pytest.mark.parametrize("behind", ["plain", "norms", "stack"])
def test_an_output_overwritten_before_the_next_models_backward(lib, behind):
    """The rows that a second model holds as its input are the first one's buffer: when that runs again the second one's backward
    would read other rows."""
    first, _ = _model("norms")
    second, _ = _model(behind)
    dout = _rows(5)
    second.forward(first.forward(_rows()))
    second.backward(dout)
    first.forward(_rows(6))
    with pytest.raises(RuntimeError, match="in place"):
        second.backward(dout)
    with torch.inference_mode():
        first.forward(_rows(7))
    first.forward(_rows(7))


@pytest.mark.parametrize("kind", ["plain", "norms", "stack"])
def test_experts_that_ran_for_someone_else(lib, kind):
    """The experts' buffers hold their last run: by itself, or for another block that shares them."""
    model, blocks = _model(kind)
    x, dout = _rows(), _rows(5)
    b = blocks[-1]
    other = MoEBlock(b.gamma.clone(), torch.zeros_like(b.gamma), b.w_router.clone(), b.experts, k)
    for use in (lambda: b.experts.forward(_rows(8, 7), *(torch.zeros(7, 1, dtype=t, device="cuda") for t in (torch.int32, torch.float32))),
                lambda: other.forward(_rows(8))):
        model.forward(x)
        use()
        with pytest.raises(RuntimeError, match="experts"):
            model.backward(dout)
        model.forward(x)
        model.backward(dout)
        model.backward(dout)
