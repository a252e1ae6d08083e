"""The residual join with outputs over its inputs at every kind of layout, wide rows with RMS norms among them, whose
reductions put no barrier between the store of r and its reads. Equal bit for bit to the call with buffers of its own."""
import pytest
import torch

from test_gpu_residual_norm import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("post,pre", [("none", "rms"), ("rms", "rms"), ("layer", "layer"), ("rms", "none")])
@pytest.mark.parametrize("stream,branch", [("fp32", "fp32"), ("fp32", "bf16"), ("bf16", "bf16")])
@pytest.mark.parametrize("T,d", [(3, 8200), (700, 8193), (2, 20001), (33, 1001), (5, 2048)])
def test_outputs_over_inputs(lib, T, d, stream, branch, post, pre):
    c = Case(T, d, stream, branch, post, pre)
    r, n, s = c.forward()
    c.check_forward(r, n, s)
    x, y = c.x.clone(), c.y.clone()
    r2, n2, s2 = c.forward(r=x, n=y if pre != "none" else None, x=x, y=y)
    assert r2 is x and torch.equal(r, x) and torch.equal(s, s2) and (n is None or torch.equal(n, y))
    if stream == branch:  # r over y, n over x
        x, y = c.x.clone(), c.y.clone()
        c.forward(r=y, n=x if pre != "none" else None, x=x, y=y)
        assert torch.equal(r, y) and (n is None or torch.equal(n, x))
    want = c.backward(r, s)
    c.check_backward(r, want)
    dr, y = c.dr.clone(), c.y.clone()
    got = c.backward(r, s, dx=dr, dr=dr, dy=y, y=y)
    assert all(torch.equal(want[k], got[k]) for k in want)
    if pre != "none":
        r2, dn = r.clone(), c.dn.clone()
        got = c.backward(r2, s, dx=r2, dy=dn, dn=dn)
        assert all(torch.equal(want[k], got[k]) for k in want)
