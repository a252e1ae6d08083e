"""The pre-norm expert block, forward and backward, against an fp64 restatement under autograd, and the
4-bit expert layer against its definition.

Tolerance of the block: every output passes through at most a dozen bf16 roundings (normalised rows,
SwiGLU output, expert rows, their sum, the residual, and their gradients), each with a relative rms
below 2^-8 / sqrt(3) = 2.3e-3 of what it rounds; added as independent errors sqrt(12) * 2.3e-3 = 8e-3."""
import numpy as np
import pytest
import torch

from oracle import mx4_oracle as Q
from ragged_grouped_gemm_device_gb300 import _lib
from ragged_grouped_gemm_device_gb300.block import MoEBlock
from ragged_grouped_gemm_device_gb300.layer import ExpertLayer, Mxfp4ExpertLayer

pytestmark = pytest.mark.gpu


def _rel(got, ref):
    got, ref = got.detach().double().cpu(), ref.detach().double().cpu()
    return float((got - ref).norm() / ref.norm())


def _parameters(E, d, h, seed):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s, std=1.0: torch.randn(*s, generator=g) * std
    bf = torch.bfloat16
    return dict(gamma=1 + 0.2 * n(d), beta=0.1 * n(d), w_router=n(E, d, std=d ** -0.5),
                w_ug=n(E, 2 * h, d, std=d ** -0.5).to(bf), w_down=n(E, h, d, std=h ** -0.5).to(bf))


def _reference(p, x, mask, ids, renorm, k, eps):
    """out, loss [2] in fp64 for given expert ids (-1: not routed)."""
    n = torch.nn.functional.layer_norm(x, x.shape[1:], p["gamma"], p["beta"], eps)
    logits = n @ p["w_router"].T
    E, h = logits.shape[1], p["w_down"].shape[1]
    prob = torch.softmax(logits, 1)
    on = ids >= 0
    safe = ids.clamp(min=0)
    w = torch.where(on, prob.gather(1, safe), torch.zeros((), dtype=torch.float64))
    if renorm:
        w = torch.where(on, w / w.sum(1, keepdim=True).clamp(min=1e-300), w)
    out = x
    for e in range(E):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if t.numel() == 0:
            continue
        u = n[t] @ p["w_ug"][e].T
        y = (torch.nn.functional.silu(u[:, :h]) * u[:, h:]) @ p["w_down"][e]
        out = out.index_add(0, t, w[t, j][:, None] * y)
    live = mask.double()
    N = live.sum()
    counts = torch.bincount(ids[on], minlength=E).double()
    balance = E * (counts / (k * N) * (prob * live[:, None]).sum(0) / N).sum()
    z = (torch.logsumexp(logits, 1).square() * live).sum() / N
    return out, torch.stack([balance, z])


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k,d,h", [(70, 8, 2, 128, 96), (333, 32, 8, 512, 64), (20, 6, 1, 64, 40)])
def test_block_forward_and_backward(lib, T, E, k, d, h, renorm):
    p = _parameters(E, d, h, T + d)
    dev = {n: v.cuda() for n, v in p.items()}
    g = torch.Generator().manual_seed(1)
    x = (torch.randn(T, d, generator=g) + 0.2).to(torch.bfloat16)
    dout = torch.randn(T, d, generator=g).to(torch.bfloat16)
    mask = torch.rand(T, generator=g) > 0.15
    d_loss = torch.tensor([2.0 * T, 0.05 * T])
    block = MoEBlock(dev["gamma"], dev["beta"], dev["w_router"], ExpertLayer(dev["w_ug"], dev["w_down"]), k, renorm)
    out = block.forward(x.cuda(), mask.cuda())
    grads = block.backward(dout.cuda(), d_loss.cuda())
    assert block.experts.status.item() == 0

    ref = {n: v.double().requires_grad_(True) for n, v in p.items()}
    xr = x.double().requires_grad_(True)
    ids = block.ids.cpu().long()
    assert torch.equal((ids >= 0).all(1), mask) and torch.equal((ids >= 0).any(1), mask)
    rout, rloss = _reference(ref, xr, mask, ids, renorm, k, block.eps)
    (rout * dout.double()).sum().add((rloss * d_loss.double()).sum()).backward()
    assert _rel(out, rout) <= 8e-3 and torch.equal(out.cpu()[~mask], x[~mask])
    assert _rel(block.loss, rloss) <= 8e-3
    want = dict(dx=xr.grad, **{n: ref[n].grad for n in p})
    for name in ("dx", "gamma", "beta", "w_router", "w_ug", "w_down"):
        assert _rel(grads[name], want[name]) <= 8e-3, name


def test_serving_block_and_4bit_training_is_refused(lib):
    T, E, k, d, h = 40, 8, 2, 256, 160
    p = {n: v.cuda() for n, v in _parameters(E, d, h, 3).items()}
    x = torch.randn(T, d, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    make = lambda experts: MoEBlock(p["gamma"], p["beta"], p["w_router"], experts, k)
    four, full = make(Mxfp4ExpertLayer(p["w_ug"], p["w_down"])), make(ExpertLayer(p["w_ug"], p["w_down"]))
    a, b = four.forward(x).clone(), full.forward(x).clone()
    assert four.experts.status.item() == 0 and torch.equal(four.ids, full.ids)
    # E2M1 steps are up to half the value below them: a 4-bit rounding is about 11% rms of what it
    # rounds, x, the weights and the SwiGLU output each once or twice
    y4, y = (a - x).double(), (b - x).double()
    assert 0.01 < float((y4 - y).norm() / y.norm()) < 0.5
    with pytest.raises(TypeError):
        four.backward(x)


@pytest.mark.parametrize("T,E,k,d,h", [(1, 16, 4, 256, 128), (50, 7, 3, 288, 160), (600, 4, 2, 128, 96)])
def test_4bit_layer_against_its_definition(lib, T, E, k, d, h):
    """The library's tolerance of a layer (5e-3): the sum of a token's expert rows is rounded as in the BF16
    layer; a code of the SwiGLU output may differ where a value lies on a rounding boundary to within
    fp32, a share of about 1e-5 of the codes, which adds below 1e-3."""
    p = _parameters(E, d, h, T + h)
    rng = np.random.default_rng(T)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    ids[rng.random((T, k)) < 0.1] = -1
    weights = rng.random((T, k)).astype(np.float32)
    x = torch.randn(T, d, generator=torch.Generator().manual_seed(T)).to(torch.bfloat16)
    layer = Mxfp4ExpertLayer(p["w_ug"].cuda(), p["w_down"].cuda())
    out = layer.forward(x.cuda(), torch.from_numpy(ids).cuda(), torch.from_numpy(weights).cuda())
    assert layer.status.item() == 0
    ref = np.zeros((T, d))
    xq = Q.fake_quant(x.double().numpy())
    for e in range(E):
        t, j = np.nonzero(ids == e)
        if t.size == 0:
            continue
        a = Q.swiglu_rows(xq[t], Q.fake_quant(p["w_ug"][e].double().numpy()))
        y = Q.fake_quant(a) @ Q.fake_quant(p["w_down"][e].double().numpy().T).T
        np.add.at(ref, t, weights[t, j][:, None] * y)
    got = out.double().cpu().numpy()
    assert np.linalg.norm(got - ref) <= 5e-3 * np.linalg.norm(ref)
    again = layer.forward(x.cuda(), torch.from_numpy(ids).cuda(), torch.from_numpy(weights).cuda())
    assert np.array_equal(again.double().cpu().numpy(), got)
    assert (got[(ids < 0).all(1)] == 0).all()


def test_the_step_in_a_graph(lib):
    """The whole serving step captured once and replayed on new inputs."""
    T, E, k, d, h = 16, 16, 4, 256, 128
    p = {n: v.cuda() for n, v in _parameters(E, d, h, 9).items()}
    block = MoEBlock(p["gamma"], p["beta"], p["w_router"], Mxfp4ExpertLayer(p["w_ug"], p["w_down"]), k)
    x = torch.empty(T, d, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(1))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        block.forward(x)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out = block.forward(x)
    for seed in (5, 6):
        x.normal_(generator=torch.Generator("cuda").manual_seed(seed))
        graph.replay()
        got = out.clone()
        assert torch.equal(got, block.forward(x))
