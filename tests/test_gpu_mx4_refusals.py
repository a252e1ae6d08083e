"""Refusals of the MXFP4 calls by both bindings (the compiled one and the ctypes functions that it replaces): every
argument with a type or a size that the kernels would read past or misread is refused before a launch."""
import pytest
import torch

from ragged_grouped_gemm_device_gb300 import _lib
from ragged_grouped_gemm_device_gb300.layer import Mxfp4ExpertLayer
from test_mx4_arguments import BF, E, F32, I32, NAMES, T, U8, _args, cap, d, h, k  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", NAMES)
def test_types_and_sizes_are_refused(lib, name):
    sizes, typed, raw = _args()[name]
    good = {n: torch.zeros(c, dtype=t, device="cuda") for n, c, t in typed + raw}
    if "offsets" in good:
        good["offsets"].fill_(cap)
    if "inv_map" in good:
        good["inv_map"].copy_(torch.arange(T * k, device="cuda"))
    for call in {getattr(_lib, name), _lib.PYTHON_BINDING.get(name, getattr(_lib, name))}:
        call(**sizes, **good)
        for n, c, t in typed:
            wrong = [good[n][:-1]] + [torch.zeros(c, dtype=o, device="cuda") for o in (F32, torch.int64, U8, torch.float16)]
            for bad in wrong + [good[n].cpu(), torch.zeros(2 * c, dtype=t, device="cuda")[::2] if c > 1 else good[n].cpu()]:
                with pytest.raises(ValueError):
                    call(**sizes, **{**good, n: bad})
        for n, c, t in raw:
            with pytest.raises((ValueError, _lib.MoEError)):  # workspaces go with their size to the library
                call(**sizes, **{**good, n: good[n][:-1]})
            with pytest.raises(ValueError):
                call(**sizes, **{**good, n: good[n].cpu()})
    torch.cuda.synchronize()


def test_layer_refusals(lib):
    layer = Mxfp4ExpertLayer(torch.zeros(E, 2 * h, d, dtype=BF, device="cuda"), torch.zeros(E, h, d, dtype=BF, device="cuda"))
    x, ids = torch.ones(T, d, dtype=BF, device="cuda"), torch.zeros(T, k, dtype=I32, device="cuda")
    w = torch.ones(T, k, device="cuda")
    assert (layer.forward(x, ids, w) == 0).all()
    good = dict(x=x, ids=ids, weights=w)
    bad = dict(x=[x.float(), x[:-1], x[:, :-32], x[0]], ids=[ids.long(), ids[:-1], ids[0]],
               weights=[w.double(), w.to(BF), w[:-1], w[:, :-1]])
    for n, values in bad.items():
        for v in values:
            with pytest.raises(ValueError):
                layer.forward(**{**good, n: v})
    with pytest.raises(ValueError):
        layer.forward(x.cpu(), ids, w)
