"""How MoEBlock behaves in a user's program beside its numbers: under autograd and with inputs that change."""
import pytest
import torch

from ragged_grouped_gemm_device_gb300.block import MoEBlock
from ragged_grouped_gemm_device_gb300.layer import ExpertLayer

pytestmark = pytest.mark.gpu

T, E, k, d, h = 24, 6, 2, 64, 40


def _block(parameters=False):
    g = torch.Generator("cuda").manual_seed(1)
    n = lambda *s, dtype=torch.float32: torch.randn(*s, generator=g, device="cuda").to(dtype)
    wrap = torch.nn.Parameter if parameters else (lambda t: t)
    w = [wrap(t) for t in (1 + 0.2 * n(d), 0.1 * n(d), n(E, d) / 8)]
    experts = ExpertLayer(n(E, 2 * h, d, dtype=torch.bfloat16) / 8, n(E, h, d, dtype=torch.bfloat16) / 6)
    return MoEBlock(*w, experts, k), n(T, d, dtype=torch.bfloat16), n(T, d, dtype=torch.bfloat16)


def test_no_partial_autograd_history(lib):
    """An output with the history of the residual alone would give x a gradient without the experts'."""
    block, x, _ = _block()
    want = block.forward(x)
    out = block.forward(x.clone().requires_grad_(True))
    assert torch.equal(out, want) and not out.requires_grad
    with pytest.raises(RuntimeError):
        out.sum().backward()


def test_weights_that_are_parameters(lib):
    block, x, dout = _block()
    want, grads = block.forward(x).clone(), {n: g.clone() for n, g in block.backward(dout).items()}
    block, _, _ = _block(parameters=True)
    assert torch.equal(block.forward(x), want)
    got = block.backward(dout)
    assert all(torch.equal(got[n], grads[n]) and not got[n].requires_grad for n in grads)


@pytest.mark.parametrize("which", ["x", "gamma", "w_router"])
def test_inputs_changed_before_the_backward(lib, which):
    """The backward reads x, gamma and w_router again: after a change in place its gradients would be those of
    another forward."""
    block, x, dout = _block()
    block.forward(x)
    {"x": x, "gamma": block.gamma, "w_router": block.w_router}[which].mul_(2.0)
    with pytest.raises(RuntimeError, match="in place"):
        block.backward(dout)
    block.forward(x)
    block.backward(dout)
    with torch.inference_mode():  # tensors without a count of changes
        block.forward(x.clone())
        block.backward(dout)


def test_refusals(lib):
    """What the experts' calls would read by its address alone is checked here: a gradient of another type or with
    fewer rows, tokens of another width or type, a mask of another length."""
    block, x, dout = _block()
    block.forward(x)
    for bad in (dout.float(), dout.half(), dout[:-1], dout[:, :-8], dout[0], dout.cpu()):
        with pytest.raises(ValueError):
            block.backward(bad)
    block.backward(dout[:1].expand(T, d))
    for bad in (x.float(), x[:, :-8], x[0], x.cpu()):
        with pytest.raises(ValueError):
            block.forward(bad)
    mask = torch.ones(T, dtype=torch.bool, device="cuda")
    for bad in (mask[:-1], torch.ones(T + 1, dtype=torch.bool, device="cuda"), mask[None], mask.float()):
        with pytest.raises(ValueError):
            block.forward(x, bad)
    block.forward(x, mask.byte())


def test_views_of_weights_follow_their_updates(lib):
    """Weights given as strided views: an update of what they view is seen by the next call."""
    block, x, dout = _block()
    stored = [torch.stack([block.gamma, block.beta], 1), block.w_router.t().contiguous()]  # [d, 2], [d, E]
    views = (stored[0][:, 0], stored[0][:, 1], stored[1].t())
    viewing = MoEBlock(*views, block.experts, k)
    viewing.forward(x)
    viewing.backward(dout)
    for t in stored:
        t.mul_(0.75).add_(0.01)
    fresh = MoEBlock(*(v.contiguous() for v in views), block.experts, k)
    want, grads = fresh.forward(x).clone(), {n: g.clone() for n, g in fresh.backward(dout).items()}
    assert not torch.equal(want, block.forward(x))
    got, now = viewing.forward(x), viewing.backward(dout)
    # the router's product may sum in another order for another layout: fp32 sums of d terms, bf16 rows
    close = lambda a, b: float((a.double() - b.double()).norm()) <= 1e-3 * float(b.double().norm())
    assert close(got, want) and all(close(now[n], grads[n]) for n in grads)
