"""A step captured into a graph goes on to use the buffers that it was captured with, also after calls of other sizes have put others
in their place: nothing else may be given that memory, and a replay gives what an eager call gives."""
import pytest
import torch

from ragged_grouped_gemm_device_gb300.block import MoEBlock, MoEStack
from ragged_grouped_gemm_device_gb300.layer import ExpertLayer, Int4ExpertLayer, Mxfp4ExpertLayer

pytestmark = pytest.mark.gpu
E, k, d, h = 6, 2, 256, 128


def _weights(seed):
    g = torch.Generator("cuda").manual_seed(seed)
    n = lambda *s, dtype=torch.float32: (torch.randn(*s, generator=g, device="cuda") / 12).to(dtype)
    return n(E, 2 * h, d, dtype=torch.bfloat16), n(E, h, d, dtype=torch.bfloat16), n


def _layer(kind, seed=1):
    ug, down, _ = _weights(seed)
    return {"bf16": ExpertLayer, "mxfp4": Mxfp4ExpertLayer, "int4": Int4ExpertLayer}[kind](ug, down)


def _block(kind, seed, plain):
    _, _, n = _weights(seed)
    if plain:
        return MoEBlock(1 + n(d), n(d), n(E, d), _layer(kind, seed), k)
    return MoEBlock(1 + n(d), None, n(E, d), _layer(kind, seed), k, pre="rms", post="rms", post_gamma=1 + n(d))


def _buffers(*owners):
    return {t.data_ptr(): t.numel() * t.element_size() for o in owners for t in vars(o).values()
            if isinstance(t, torch.Tensor) and t.is_cuda and t.numel() > 0}


@pytest.mark.parametrize("what", ["bf16", "mxfp4", "int4", "plain block", "stack of bf16", "stack of int4"])
def test_calls_of_another_size_between_capture_and_replay(lib, what):
    g = torch.Generator("cuda").manual_seed(9)
    rows = lambda T: torch.randn(T, d, generator=g, device="cuda").bfloat16()
    back = False
    if what in ("bf16", "mxfp4", "int4"):
        layer = _layer(what)
        owners = [layer]
        route = {T: (torch.randint(0, E, (T, k), dtype=torch.int32).cuda(), torch.rand(T, k).cuda()) for T in (40, 90)}
        step = lambda x: [layer.forward(x, *route[x.shape[0]])]
    else:
        kind = "int4" if "int4" in what else "bf16"
        blocks = [_block(kind, 3, True)] if what == "plain block" else [_block(kind, 3, True), _block(kind, 5, False)]
        model = blocks[0] if what == "plain block" else MoEStack(blocks)
        owners = [o for b in blocks for o in (b, b.experts)] + [getattr(model, "_joins", None) or model]
        back = kind == "bf16"

        def step(x):
            out = [model.forward(x)]
            if back:
                got = model.backward(x)
                out += [got["dx"]] + [t for part in got.get("blocks", [got]) for _, t in sorted(part.items())]
            return out
    x = rows(40)
    step(x)                                              # the buffers of these sizes are from before the capture
    held = _buffers(*owners)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = step(x)
    step(rows(90))
    torch.cuda.synchronize()
    others = [torch.full((n,), 77, dtype=torch.uint8, device="cuda") for n in held.values() for _ in range(2)]
    spans = [(t.data_ptr(), t.data_ptr() + t.numel()) for t in others]
    assert not any(a < p + n and p < b for a, b in spans for p, n in held.items())
    x.copy_(rows(40))
    graph.replay()
    got = [t.clone() for t in out]
    assert all(torch.equal(a, b) for a, b in zip(got, step(x)))
    assert all((t == 77).all() for t in others)
