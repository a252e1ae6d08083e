"""Blocks with norms on both sides, a stack of them, and a run as a user's program makes it: train the stack with AdamW,
then serve it on 4-bit weights.

Tolerance of the stack against fp64 under autograd: as for the block (sqrt of the number of bf16 roundings that an output passes,
each at most 2^-8 / sqrt(3)): a dozen a block, so sqrt(24) * 2.3e-3 = 1.1e-2 for two."""
import pytest
import torch

from ragged_grouped_gemm_device_gb300 import _lib
from ragged_grouped_gemm_device_gb300.block import MoEBlock, MoEStack
from ragged_grouped_gemm_device_gb300.layer import ExpertLayer, Int4ExpertLayer, Mxfp4ExpertLayer
from ragged_grouped_gemm_device_gb300.optim import AdamW

pytestmark = pytest.mark.gpu
E, d, h, k = 6, 128, 48, 2


def _rel(got, ref):
    got, ref = got.detach().double().cpu(), ref.detach().double().cpu()
    return float((got - ref).norm() / ref.norm())


def _parameters(seed, pre, post):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s, std=1.0: torch.randn(*s, generator=g) * std
    bf = torch.bfloat16
    p = dict(gamma=1 + 0.2 * n(d), w_router=n(E, d, std=d ** -0.5), gate=0.5 + 0.2 * n(d),
             w_ug=n(E, 2 * h, d, std=d ** -0.5).to(bf), w_down=n(E, h, d, std=h ** -0.5).to(bf))
    if pre == "layer":
        p["beta"] = 0.1 * n(d)
    if post != "none":
        p["post_gamma"] = 1 + 0.2 * n(d)
    if post == "layer":
        p["post_beta"] = 0.1 * n(d)
    return p


def _block(p, pre, post, experts=None, res=0.8, branch=0.6):
    c = {n: t.cuda() for n, t in p.items()}
    experts = experts or ExpertLayer(c["w_ug"], c["w_down"])
    return MoEBlock(c["gamma"], c.get("beta"), c["w_router"], experts, k, pre=pre, post=post, post_gamma=c.get("post_gamma"),
                    post_beta=c.get("post_beta"), gate=c["gate"], res_scale=res, branch_scale=branch)


def _norm(kind, x, gamma, beta, eps=1e-5):
    if kind == "none":
        return x
    c = x - x.mean(1, keepdim=True) if kind == "layer" else x
    y = c / (c.square().mean(1, keepdim=True) + eps).sqrt() * gamma
    return y if beta is None else y + beta


def _reference(p, x, ids, pre, post, res=0.8, branch=0.6):
    n = _norm(pre, x, p["gamma"], p.get("beta"))
    w = torch.softmax(n @ p["w_router"].T, 1).gather(1, ids.clamp(min=0)) * (ids >= 0)
    w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    y = torch.zeros_like(x)
    for e in range(E):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        u = n[t] @ p["w_ug"][e].T
        y = y.index_add(0, t, w[t, j][:, None] * ((torch.nn.functional.silu(u[:, :h]) * u[:, h:]) @ p["w_down"][e]))
    return res * x + branch * p["gate"] * _norm(post, y, p.get("post_gamma"), p.get("post_beta"))


KINDS = [("rms", "rms"), ("layer", "layer"), ("rms", "none")]


@pytest.mark.parametrize("pre,post", KINDS)
@pytest.mark.parametrize("count", [1, 2])
def test_gradients_against_fp64(lib, pre, post, count):
    T = 90
    ps = [_parameters(10 + i, pre, post) for i in range(count)]
    blocks = [_block(p, pre, post) for p in ps]
    g = torch.Generator().manual_seed(1)
    x, dout = (torch.randn(T, d, generator=g) + 0.2).bfloat16(), torch.randn(T, d, generator=g).bfloat16()
    mask = torch.rand(T, generator=g) > 0.1
    model = MoEStack(blocks) if count > 1 else blocks[0]
    out = model.forward(x.cuda(), mask.cuda()).clone()
    got = model.backward(dout.cuda())
    grads = got["blocks"] if count > 1 else [got]
    refs = [{n: t.double().requires_grad_(True) for n, t in p.items()} for p in ps]
    xr = r = x.double().requires_grad_(True)
    for b, p in zip(blocks, refs):
        ids = b.ids.cpu().long()
        assert torch.equal((ids >= 0).all(1), mask)
        r = _reference(p, r, ids, pre, post)
    (r * dout.double()).sum().backward()
    tol = 8e-3 if count == 1 else 1.1e-2
    assert _rel(out, r) <= tol and _rel(got["dx"], xr.grad) <= tol
    for b, mine, p in zip(blocks, grads, refs):
        assert set(b.tensors()) == set(p) and set(p) <= set(mine)
        for n in p:
            assert _rel(mine[n], p[n].grad) <= tol, n


def test_a_stack_is_its_blocks(lib):
    """The fused joins give what the calls between the blocks give by themselves, forward and backward, bit for bit: r
    and the rows of both norms are rounded once wherever they are computed. (dx takes one rounding less in the
    stack.)"""
    T = 77
    g = torch.Generator("cuda").manual_seed(4)
    x = torch.randn(T, d, generator=g, device="cuda").bfloat16()
    ps = [_parameters(20 + i, "rms", "layer") for i in range(3)]
    alone, stack = [_block(p, "rms", "layer") for p in ps], MoEStack([_block(p, "rms", "layer") for p in ps])
    r = x
    for b in alone:
        r = b.forward(r).clone()
    out = stack.forward(x)
    assert torch.equal(out, r)
    dout = torch.randn(T, d, generator=g, device="cuda").bfloat16()
    got = stack.backward(dout, [None, torch.tensor([1.0, 0.1], device="cuda"), None])
    last = alone[2].backward(dout)
    for n in ("w_ug", "w_down", "w_router", "post_gamma", "post_beta", "gate"):
        assert torch.equal(got["blocks"][2][n], last[n]), n
    again = {n: t.clone() for n, t in got["blocks"][0].items()}
    stack.forward(x)
    repeat = stack.backward(dout, [None, torch.tensor([1.0, 0.1], device="cuda"), None])
    assert all(torch.equal(again[n], repeat["blocks"][0][n]) for n in again)


def test_default_block_is_unchanged(lib):
    """Without the new arguments a block is layer norm, experts and a bf16 addition, as before."""
    p = {n: t.cuda() for n, t in _parameters(3, "layer", "none").items()}
    block = MoEBlock(p["gamma"], p["beta"], p["w_router"], ExpertLayer(p["w_ug"], p["w_down"]), k)
    x = torch.randn(40, d, device="cuda").bfloat16()
    out = block.forward(x)
    assert torch.equal(out, x + block.experts.out)
    n = torch.empty_like(x)
    _lib.moe_layer_norm_fwd(x, p["gamma"], p["beta"], 40, d, block.eps, n)
    assert torch.equal(n, block.normed)


@pytest.mark.parametrize("state_bits", [32, 8])
def test_train_then_serve(lib, state_bits):
    """Several steps of training move every tensor and keep everything finite; the trained stack served on 4-bit weights, one
    token after another, gives the rows of the BF16 stack to the weights' rounding."""
    T = 64
    ps = [_parameters(30 + i, "rms", "rms") for i in range(2)]
    blocks = [_block(p, "rms", "rms", res=1.0, branch=1.0) for p in ps]
    stack = MoEStack(blocks)
    names = [(i, n) for i, b in enumerate(blocks) for n in b.tensors()]
    tensors = [blocks[i].tensors()[n] for i, n in names]
    # fp32 master weights of the experts, whose bf16 weights the products read
    masters = [t.float() if t.dtype == torch.bfloat16 else t for t in tensors]
    copies = [t if t.dtype == torch.bfloat16 else None for t in tensors]
    before = [t.clone() for t in tensors]
    opt = AdamW(masters, lr=1e-2, betas=(0.9, 0.95), weight_decay=0.1, state_bits=state_bits, copies=copies, max_norm=1.0)
    g = torch.Generator("cuda").manual_seed(8)
    x = torch.randn(T, d, generator=g, device="cuda").bfloat16()
    target = torch.randn(T, d, generator=g, device="cuda").bfloat16()
    for _ in range(4):
        out = stack.forward(x)
        grads = stack.backward(out - target, [torch.full((2,), 0.01, device="cuda")] * 2)["blocks"]
        norm = opt.step([grads[i][n] for i, n in names])
        with pytest.raises(RuntimeError, match="in place"):                  # the step changed what the backward reads
            stack.backward(out - target)
    assert opt.steps == 4 and torch.isfinite(norm)
    assert all(torch.isfinite(t).all() and not torch.equal(t, b) for t, b in zip(tensors, before))
    assert all(torch.equal(c, m.bfloat16()) for m, c in zip(masters, copies) if c is not None)

    full = stack.forward(x).clone()
    serve = []
    for b in blocks:
        c = {n: t for n, t in b.tensors().items()}
        serve.append(MoEBlock(c["gamma"], None, c["w_router"], Int4ExpertLayer(c["w_ug"], c["w_down"], 32), k, pre="rms", post="rms",
                              post_gamma=c["post_gamma"], gate=c["gate"]))
    four = MoEStack(serve)
    whole = four.forward(x).clone()
    # a 4-bit step of a group of 32 is about a seventh of its largest value, 0.3 of a deviation: a rounding of 0.09, three times;
    # behind the norm and a gate near a half beside the residual
    assert 1e-3 < _rel(whole, full) < 0.25
    rows = torch.cat([four.forward(x[t:t + 1]).clone() for t in range(8)])
    # alone or in a batch: other sums of the same terms, and roundings that they move by a place
    assert _rel(rows, whole[:8]) < 1.1e-2
    with pytest.raises(TypeError):
        four.backward(x)


def test_serving_step_in_a_graph(lib):
    blocks = []
    for i, kind in enumerate((Int4ExpertLayer, Mxfp4ExpertLayer)):
        p = _parameters(40 + i, "rms", "none")
        p["w_ug"], p["w_down"] = torch.randn(E, 64, d).bfloat16() * d ** -0.5, torch.randn(E, 32, d).bfloat16() * 32 ** -0.5
        blocks.append(_block(p, "rms", "none", kind(p["w_ug"].cuda(), p["w_down"].cuda())))
    stack = MoEStack(blocks)
    x = torch.randn(3, d, device="cuda").bfloat16()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        stack.forward(x)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = stack.forward(x)
    for _ in range(2):
        x.normal_()
        graph.replay()
        got = out.clone()
        assert torch.equal(got, stack.forward(x))


def test_refusals(lib):
    p = _parameters(5, "rms", "rms")
    a, b = _block(p, "rms", "rms"), _block(p, "rms", "rms")
    for bad in ([], [a, a], [a, _block(p, "rms", "rms", experts=a.experts)]):
        with pytest.raises(ValueError):
            MoEStack(bad)
    stack = MoEStack([a, b])
    x = torch.randn(5, d, device="cuda").bfloat16()
    with pytest.raises(RuntimeError):
        stack.backward(x)
    for bad in (x.float(), x[:, :64], x.cpu()):
        with pytest.raises(ValueError):
            stack.forward(bad)
    with pytest.raises(ValueError):
        stack.forward(x, torch.ones(4, dtype=torch.bool, device="cuda"))
    stack.forward(x)
    with pytest.raises(ValueError):
        stack.backward(x, [None])
    with pytest.raises(ValueError):
        stack.backward(x[:4])
    a.gate.mul_(2.0)
    with pytest.raises(RuntimeError, match="in place"):
        stack.backward(x)
    # one eps for the norms on both sides of a join
    b.eps = 1e-3
    with pytest.raises(ValueError, match="eps"):
        MoEStack([a, b])
    MoEStack([b])
    for bad in (dict(pre="none"), dict(post="norm"), dict(post="none"), dict(post="rms", post_beta=a.gate)):
        with pytest.raises(AssertionError):
            MoEBlock(**{**dict(gamma=a.gamma, beta=None, w_router=a.w_router, experts=a.experts, top_k=2, pre="rms", post="rms", post_gamma=a.gate), **bad})


def test_backward_of_a_run_that_is_gone(lib):
    """A block's buffers hold its last run, whoever asked for it."""
    p, q = _parameters(5, "rms", "rms"), _parameters(6, "layer", "none")
    a, b = _block(p, "rms", "rms"), _block(p, "rms", "rms")
    plain = MoEBlock(*(q[n].cuda() for n in ("gamma", "beta", "w_router")), ExpertLayer(q["w_ug"].cuda(), q["w_down"].cuda()), k)
    stack, x = MoEStack([plain, a, b]), torch.randn(5, d, device="cuda").bfloat16()
    with pytest.raises(RuntimeError):
        plain.backward(x)
    for alone in (plain, a):
        stack.forward(x)
        with pytest.raises(RuntimeError):
            alone.backward(x)
        alone.forward(x)
        with pytest.raises(RuntimeError, match="another"):
            stack.backward(x)
        alone.backward(x)
    MoEStack([b, a]).forward(x)
    with pytest.raises(RuntimeError, match="another"):
        stack.backward(x)
    stack.forward(x)
    stack.backward(x)
