"""Layer norm with an output in the place of an input: the same bits as with a buffer of its own."""
import pytest
import torch

from ragged_grouped_gemm_device_gb300 import _lib

pytestmark = pytest.mark.gpu


# rows in registers (one and several chunks, odd widths) and rows that are read several times
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,d", [(5000, 96), (700, 2048), (300, 1001), (40, 8200), (9, 16392), (700, 20000), (3, 40001)])
def test_outputs_over_inputs(lib, T, d, dtype):
    g = torch.Generator("cuda").manual_seed(T + d)
    n = lambda *s, dtype=torch.float32: torch.randn(*s, generator=g, device="cuda").to(dtype)
    x, dy, gamma, beta = n(T, d, dtype=dtype), n(T, d, dtype=dtype), n(d), n(d)
    mean, rstd = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    ws = torch.empty(_lib.moe_workspace_bytes(_lib.OP_LAYER_NORM_BWD, T, 1, 1, d), dtype=torch.uint8, device="cuda")

    def backward(dy, x, dx):
        dg, db = torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
        _lib.moe_layer_norm_bwd(dy, x, gamma, mean, rstd, T, d, dx, dg, db, ws)
        return dx, dg, db

    y = torch.empty_like(x)
    _lib.moe_layer_norm_fwd(x, gamma, beta, T, d, 1e-5, y, mean, rstd)
    over = x.clone()
    _lib.moe_layer_norm_fwd(over, gamma, beta, T, d, 1e-5, over)
    assert torch.equal(over, y)
    want = backward(dy, x, torch.empty_like(x))
    a, b = x.clone(), dy.clone()
    assert all(torch.equal(p, q) for p, q in zip(backward(dy, a, a), want))
    assert all(torch.equal(p, q) for p, q in zip(backward(b, x, b), want))
