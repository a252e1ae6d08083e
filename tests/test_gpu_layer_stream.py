"""The layers on a stream of their own while torch's current stream is busy: dense copies of strided inputs
belong to the layer's stream, so the results do not depend on what the current stream is doing."""
import pytest
import torch

from ragged_grouped_gemm_device_gb300.layer import ExpertLayer, Mxfp4ExpertLayer

pytestmark = pytest.mark.gpu

T, E, k, d, h = 48, 6, 2, 96, 64
BUSY = 400_000_000  # cycles of the current stream, about a fifth of a second: far longer than the calls


def _inputs():
    g = torch.Generator("cuda").manual_seed(7)
    n = lambda *s, dtype=torch.bfloat16: torch.randn(*s, generator=g, device="cuda").to(dtype)
    # views that a dense copy is made of: weights stored transposed, rows of a wider buffer
    w_ug, w_down = (n(E, d, 2 * h) / 10).transpose(1, 2), (n(E, d, h) / 8).transpose(1, 2)
    x, dout = n(T, d + 8)[:, :d], n(T, d + 8)[:, :d]
    ids = torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    return w_ug, w_down, x, dout, ids, torch.rand(T, k, generator=g, device="cuda")


def test_4bit_layer(lib):
    w_ug, w_down, x, _, ids, w = _inputs()
    want = Mxfp4ExpertLayer(w_ug, w_down).forward(x, ids, w).clone()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    layer = Mxfp4ExpertLayer(w_ug, w_down, stream=s)
    out = layer.forward(x, ids, w, stream=s)
    s.synchronize()
    assert not torch.cuda.current_stream().query()  # still busy: nothing waited for it
    with torch.cuda.stream(s):
        got = out.clone()
    assert torch.equal(got, want)
    torch.cuda.synchronize()


def test_bf16_layer(lib):
    w_ug, w_down, x, dout, ids, w = _inputs()
    layer = ExpertLayer(w_ug, w_down)
    want = [layer.forward(x, ids, w).clone()] + [t.clone() for t in layer.backward(dout)]
    layer, s = ExpertLayer(w_ug, w_down), torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    got = [layer.forward(x, ids, w, s).clone, *(t.clone for t in layer.backward(dout, s))]
    s.synchronize()
    assert not torch.cuda.current_stream().query()
    with torch.cuda.stream(s):
        got = [clone() for clone in got]
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    torch.cuda.synchronize()
