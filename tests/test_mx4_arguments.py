"""What the Python functions of the MXFP4 calls pass on (no GPU: the library and the tensors are stand-ins that only
have what a check reads). Types and sizes that the kernels would take by their address alone are refused."""
import pytest
import torch

from ragged_grouped_gemm_device_gb300 import _lib, build

BF, I32, U8, F32 = torch.bfloat16, torch.int32, torch.uint8, torch.float32


class Tensor:
    """A CUDA tensor as far as an argument check goes."""
    is_cuda = True

    def __init__(self, numel, dtype):
        self.n, self.dtype = numel, dtype

    def numel(self):
        return self.n

    def element_size(self):
        return self.dtype.itemsize

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 256


class Recorder:
    """The library with every launch replaced by a note."""

    def __init__(self, real):
        self.real, self.calls = real, []

    def __getattr__(self, name):
        if name == "moe_workspace_bytes":
            return self.real.moe_workspace_bytes
        return lambda *a: self.calls.append(name) or 0


E, T, k, d, h, cap = 5, 12, 3, 96, 64, 36
N = T * k


def _args():
    wb = _lib.moe_workspace_bytes
    scales = wb(_lib.OP_MX4_ROW_SCALES, cap, 1, E, d, 32)
    mxw = wb(_lib.OP_MX4_WEIGHTS, 0, 1, E, d, h)
    ws = wb(_lib.OP_MX4_FWD, cap, 1, E, d, h)
    st = ("dev_status", 1, I32)
    return {
        "moe_mx4_prepare_weights": (dict(E=E, d=d, h=h), [("w_ug", 2 * E * h * d, BF), ("w_down", E * h * d, BF)],
                                    [("mxw", mxw, U8)]),
        "moe_mx4_quantize_rows": (dict(E=E, cap=cap, K=d), [("x", cap * d, BF), ("offsets", E, I32), st],
                                  [("q", cap * d // 2, U8), ("sf", scales, U8)]),
        "moe_mx4_dequantize_rows": (dict(E=E, cap=cap, K=d), [("x", cap * d, BF), ("offsets", E, I32), st],
                                    [("q", cap * d // 2, U8), ("sf", scales, U8)]),
        "moe_permute_mxfp4": (dict(T=T, top_k=k, E=E, d=d),
                              [("x", T * d, BF), ("inv_map", N, I32), ("offsets", E, I32), st],
                              [("q", N * d // 2, U8), ("sf", scales, U8)]),
        "moe_grouped_swiglu_fwd_mxfp4": (dict(E=E, cap=cap, d=d, h=h), [("offsets", E, I32), ("y", cap * d, BF), st],
                                         [("xq", cap * d // 2, U8), ("xsf", scales, U8), ("mxw", mxw, U8), ("ws", ws, U8)]),
    }


NAMES = ["moe_mx4_prepare_weights", "moe_mx4_quantize_rows", "moe_mx4_dequantize_rows", "moe_permute_mxfp4",
         "moe_grouped_swiglu_fwd_mxfp4"]


@pytest.mark.parametrize("name", NAMES)
def test_types_and_sizes_are_checked(name, monkeypatch):
    build.build()
    fake = Recorder(_lib.load())
    monkeypatch.setattr(_lib, "load", lambda: fake)
    monkeypatch.setattr(_lib, "_stream", lambda s: 0)
    call = _lib.PYTHON_BINDING.get(name, getattr(_lib, name))
    sizes, typed, raw = _args()[name]
    good = {n: Tensor(c, t) for n, c, t in typed + raw}
    call(**sizes, **good)
    assert fake.calls == [name]
    for n, c, t in typed:
        wrong = [Tensor(c - 1, t)] + [Tensor(c, o) for o in (F32, torch.int64, U8, torch.float16)]
        for bad in wrong:
            with pytest.raises(ValueError):
                call(**sizes, **{**good, n: bad})
        if n == "dev_status":
            call(**sizes, **{**good, n: None})
    fake.calls.clear()
    for n, c, t in raw:
        call(**sizes, **{**good, n: Tensor(c, torch.int8)})             # bytes are bytes
        call(**sizes, **{**good, n: Tensor((c + 3) // 4, F32)})
        if n not in ("ws", "mxw") or name == "moe_grouped_swiglu_fwd_mxfp4" and n == "mxw":
            before = len(fake.calls)
            with pytest.raises(ValueError):
                call(**sizes, **{**good, n: Tensor(c - 1, U8)})         # (ws and the weights' buffer go with their size)
            assert len(fake.calls) == before


def test_no_rows_need_no_buffers(monkeypatch):
    """cap = 0 with empty tensors passes the checks, as the library allows."""
    build.build()
    fake = Recorder(_lib.load())
    monkeypatch.setattr(_lib, "load", lambda: fake)
    monkeypatch.setattr(_lib, "_stream", lambda s: 0)
    binding = lambda n: _lib.PYTHON_BINDING.get(n, getattr(_lib, n))
    none = lambda t: Tensor(0, t)
    off = Tensor(E, I32)
    binding("moe_mx4_quantize_rows")(none(BF), off, E, 0, d, none(U8), none(U8))
    binding("moe_mx4_dequantize_rows")(none(U8), none(U8), off, E, 0, d, none(BF))
    binding("moe_permute_mxfp4")(none(BF), none(I32), off, 0, k, E, d, none(U8), none(U8))
    mxw = Tensor(_lib.moe_workspace_bytes(_lib.OP_MX4_WEIGHTS, 0, 1, E, d, h), U8)
    binding("moe_grouped_swiglu_fwd_mxfp4")(none(U8), none(U8), off, E, 0, d, h, mxw, none(BF), none(U8))
    assert len(fake.calls) == 4
