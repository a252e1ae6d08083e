"""A block or stack that nobody holds any longer is gone at once, with its weights and buffers: nothing in it refers back to it, or
its memory on the GPU would wait for the garbage collector, which does not know of it."""
import copy
import gc
import weakref

import pytest
import torch

from ragged_grouped_gemm_device_gb300.block import MoEBlock, MoEStack
from ragged_grouped_gemm_device_gb300.layer import ExpertLayer

T, E, k, d, h = 16, 4, 2, 64, 40


def _block(device, plain):
    n = lambda *s, dtype=torch.float32: (torch.randn(*s, device=device) / 8).to(dtype)
    experts = ExpertLayer(n(E, 2 * h, d, dtype=torch.bfloat16), n(E, h, d, dtype=torch.bfloat16))
    if plain:
        return MoEBlock(n(d), n(d), n(E, d), experts, k)
    return MoEBlock(n(d), None, n(E, d), experts, k, pre="rms", post="rms", post_gamma=n(d))


@pytest.fixture
def no_gc():
    gc.collect()
    gc.disable()
    yield
    gc.enable()


@pytest.mark.parametrize("plain", [True, False])
def test_a_block_that_has_not_run(no_gc, plain):
    block = _block("cpu", plain)
    gone = [weakref.ref(block), weakref.ref(block.experts)]
    del block
    assert all(r() is None for r in gone)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["plain", "norms", "stack"])
def test_what_has_run(lib, no_gc, kind):
    x = torch.randn(T, d, device="cuda").bfloat16()
    torch.cuda.synchronize()
    for turn in range(2):                      # what the first call leaves in libraries for good is there in the second
        before = torch.cuda.memory_allocated()
        blocks = [_block("cuda", kind == "plain")] if kind != "stack" else [_block("cuda", True), _block("cuda", False)]
        model = MoEStack(blocks) if kind == "stack" else blocks[0]
        model.forward(x)
        model.backward(x)
        gone = [weakref.ref(b) for b in blocks]
        del model, blocks
        assert all(r() is None for r in gone)
    assert torch.cuda.memory_allocated() == before


@pytest.mark.gpu
def test_a_copy_is_a_block_of_its_own(lib):
    x = torch.randn(T, d, device="cuda").bfloat16()
    for plain in (True, False):
        block = _block("cuda", plain)
        want = block.forward(x).clone()
        other = copy.deepcopy(block)
        other.experts.w_down.zero_()
        assert not torch.equal(other.forward(x), want) and torch.equal(block.forward(x), want)
        block.backward(x)
