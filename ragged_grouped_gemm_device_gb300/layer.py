"""One SwiGLU expert layer driven through the C ABI: route -> permute -> grouped forward ->
combine, and the backward pass. PyTorch only allocates device memory and supplies the stream;
every step is a library kernel. Buffers are allocated once per shape and reused, so repeated
calls with new routing allocate nothing ("Section 09: Grouped GEMM" §9.4: fixed physical
shapes, unpadded compute)."""
from __future__ import annotations

import contextlib

import torch

from . import _lib


def _dense(t: torch.Tensor) -> torch.Tensor:
    """The library reads row-major contiguous rows. A view with other strides -- notably the
    zero-stride gradient a scalar loss broadcasts back (`out.sum().backward()` hands over an
    expanded [T, d] tensor with strides (0, 0)), which "Grouped expert GEMM" lists as an edge case
    of the grouped GEMM's backward -- is materialised once here; dense tensors pass through."""
    return t if t.is_contiguous() else t.contiguous()


def _on(stream):
    """`stream` (nullable) as torch's current one, for the dense copies and buffers of a call whose kernels run
    on it: a copy made on another stream would be read before it is written, and its memory given away
    while it is still read. The caller's own tensors have to be ready on `stream`."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


class ExpertLayer:
    """Holds the expert weights W_ug [E, 2h, d] and W_down [E, h, d] (bf16, on the device)."""

    def __init__(self, w_ug: torch.Tensor, w_down: torch.Tensor):
        E, two_h, d = w_ug.shape
        assert w_down.shape == (E, two_h // 2, d)
        assert w_ug.dtype == torch.bfloat16 and w_down.dtype == torch.bfloat16
        self.E, self.d, self.h = E, d, two_h // 2
        self.w_ug, self.w_down = w_ug.contiguous(), w_down.contiguous()
        self.device = w_ug.device
        self._key = None
        self.status = torch.zeros(1, dtype=torch.int32, device=self.device)

    def _buffers(self, T: int, k: int):
        if self._key == (T, k):
            return
        dev, E, d, h, n = self.device, self.E, self.d, self.h, T * k
        i32, bf = torch.int32, torch.bfloat16
        self.counts = torch.empty(E, dtype=i32, device=dev)
        self.offsets = torch.empty(E, dtype=i32, device=dev)
        self.sorted_src = torch.empty(max(n, 1), dtype=i32, device=dev)
        self.inv_map = torch.empty(max(n, 1), dtype=i32, device=dev)
        rw = _lib.moe_workspace_bytes(_lib.OP_ROUTE, T, k, E, d, h)
        self.route_ws = torch.empty(max(rw, 1), dtype=torch.uint8, device=dev)
        self.xp = torch.empty(max(n, 1), d, dtype=bf, device=dev)
        self.y = torch.empty(max(n, 1), d, dtype=bf, device=dev)
        self.a = torch.empty(max(n, 1), h, dtype=bf, device=dev)
        sv = _lib.moe_workspace_bytes(_lib.OP_SAVED, T, k, E, d, h)
        self.saved = torch.empty(max(sv, 1), dtype=torch.uint8, device=dev)
        self.out = torch.empty(T, d, dtype=bf, device=dev)
        self.dy = torch.empty(max(n, 1), d, dtype=bf, device=dev)
        self.dxp = torch.empty(max(n, 1), d, dtype=bf, device=dev)
        self.dx = torch.empty(T, d, dtype=bf, device=dev)
        self.dw_ug = torch.empty(E, 2 * h, d, dtype=torch.float32, device=dev)
        self.dw_down = torch.empty(E, h, d, dtype=torch.float32, device=dev)
        self.dw_route = torch.empty(T, k, dtype=torch.float32, device=dev)
        fw = _lib.moe_workspace_bytes(_lib.OP_FWD, T, k, E, d, h)
        self.fwd_ws = torch.empty(fw, dtype=torch.uint8, device=dev) if fw > 0 else None
        bw = _lib.moe_workspace_bytes(_lib.OP_BWD, T, k, E, d, h)
        self.bwd_ws = torch.empty(max(bw, 1), dtype=torch.uint8, device=dev)
        self._key = (T, k)

    def forward(self, x: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, stream=None):
        """x [T, d] bf16, ids [T, k] int32, weights [T, k] fp32 -> out [T, d] bf16."""
        T, k = ids.shape
        with _on(stream):
            x, ids, weights = _dense(x), _dense(ids), _dense(weights)
            self._buffers(T, k)
        self.T, self.k, self.weights = T, k, weights
        E, d, h, n = self.E, self.d, self.h, T * k
        _lib.moe_route_offsets(ids, T, k, E, self.counts, self.offsets, self.sorted_src, self.inv_map,
                               self.route_ws, stream)
        _lib.moe_permute(x, self.sorted_src, self.offsets, None, T, k, E, d, self.xp, stream)
        if k == 1 and d % 8 == 0 and h % 8 == 0:
            # one slot per token: the down projection writes the token rows itself (no y, no
            # combine pass); the routing weight is folded into the SwiGLU output
            _lib.moe_grouped_swiglu_fwd_top1_combine(self.xp, self.offsets, self.sorted_src, self.inv_map, weights,
                                                     E, T, d, h, self.w_ug, self.w_down, self.out, self.a,
                                                     self.saved, self.status, stream)
            return self.out
        # the routing weight is applied in the up/gate projection's epilogue; the combine sums
        _lib.moe_grouped_swiglu_fwd(self.xp, self.offsets, self.sorted_src, weights, E, n, d, h, self.w_ug,
                                    self.w_down, self.y, self.a, self.saved, self.fwd_ws, self.status, stream)
        _lib.moe_unpermute_combine(self.y, self.inv_map, None, T, k, d, self.out, stream)
        return self.out

    def backward(self, dout: torch.Tensor, stream=None):
        """dout [T, d] bf16 -> (dx [T, d] bf16, dW_ug [E, 2h, d] fp32, dW_down [E, h, d] fp32,
        d_weights [T, k] fp32: the gradient of the routing weights, 0 for dropped slots)."""
        T, k, E, d, h, n = self.T, self.k, self.E, self.d, self.h, self.T * self.k
        with _on(stream):
            dout = _dense(dout)
        _lib.moe_permute(dout, self.sorted_src, self.offsets, None, T, k, E, d, self.dy, stream)
        _lib.moe_grouped_bwd(self.dy, self.xp, self.a, self.saved, self.offsets, self.sorted_src, self.weights,
                             E, n, d, h, self.w_ug,
                             self.w_down, self.dxp, self.dw_ug, self.dw_down, self.bwd_ws, self.status,
                             stream, inv_map=self.inv_map, dw_route=self.dw_route)
        _lib.moe_unpermute_combine(self.dxp, self.inv_map, None, T, k, d, self.dx, stream)
        return self.dx, self.dw_ug, self.dw_down, self.dw_route


class Mxfp4ExpertLayer:
    """The forward of one SwiGLU expert layer on 4-bit weights and activations (serving; no backward).

    Takes the bf16 weights of ExpertLayer, quantizes them once (`weights` holds the codes and
    scales; the bf16 tensors are not kept) and runs route -> gather + quantize -> grouped products
    -> combine. d and h multiples of 32."""

    def __init__(self, w_ug: torch.Tensor, w_down: torch.Tensor, stream=None):
        E, two_h, d = w_ug.shape
        assert w_down.shape == (E, two_h // 2, d)
        assert w_ug.dtype == torch.bfloat16 and w_down.dtype == torch.bfloat16
        self.E, self.d, self.h = E, d, two_h // 2
        self.device = w_ug.device
        n = _lib.moe_workspace_bytes(_lib.OP_MX4_WEIGHTS, 0, 1, E, d, self.h)
        with _on(stream):
            self.weights = torch.empty(max(n, 1), dtype=torch.uint8, device=self.device)
            w_ug, w_down = _dense(w_ug), _dense(w_down)
            self.status = torch.zeros(1, dtype=torch.int32, device=self.device)
        _lib.moe_mx4_prepare_weights(w_ug, w_down, E, d, self.h, self.weights, stream)
        self._key = None

    def _buffers(self, T: int, k: int):
        if self._key == (T, k):
            return
        E, d, h, n = self.E, self.d, self.h, T * k
        new = lambda *shape, dtype: torch.empty(*shape, dtype=dtype, device=self.device)  # noqa: E731
        room = lambda op: new(max(1, _lib.moe_workspace_bytes(op, T, k, E, d, h)), dtype=torch.uint8)  # noqa: E731
        self.counts, self.offsets = new(E, dtype=torch.int32), new(E, dtype=torch.int32)
        self.sorted_src, self.inv_map = new(max(n, 1), dtype=torch.int32), new(max(n, 1), dtype=torch.int32)
        self.route_ws, self.fwd_ws = room(_lib.OP_ROUTE), room(_lib.OP_MX4_FWD)
        self.xq, self.xsf = new(max(n, 1), d // 2, dtype=torch.uint8), room(_lib.OP_MX4_ROW_SCALES)
        self.y, self.out = new(max(n, 1), d, dtype=torch.bfloat16), new(T, d, dtype=torch.bfloat16)
        self._key = (T, k)

    def forward(self, x: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, stream=None):
        """x [T, d] bf16, ids [T, k] int32, weights [T, k] fp32 -> out [T, d] bf16."""
        if ids.dim() != 2 or ids.dtype != torch.int32:
            raise ValueError("ids has to be [T, k] int32")
        T, k = ids.shape
        if tuple(x.shape) != (T, self.d) or x.dtype != torch.bfloat16:
            raise ValueError(f"x has to be [{T}, {self.d}] bfloat16")
        if tuple(weights.shape) != (T, k) or weights.dtype != torch.float32:
            raise ValueError(f"weights has to be [{T}, {k}] float32")
        with _on(stream):
            x, ids, weights = _dense(x), _dense(ids), _dense(weights)
            self._buffers(T, k)
        E, d, h, n = self.E, self.d, self.h, T * k
        _lib.moe_route_offsets(ids, T, k, E, self.counts, self.offsets, self.sorted_src, self.inv_map,
                               self.route_ws, stream)
        _lib.moe_permute_mxfp4(x, self.inv_map, self.offsets, T, k, E, d, self.xq, self.xsf, self.status, stream)
        _lib.moe_grouped_swiglu_fwd_mxfp4(self.xq, self.xsf, self.offsets, E, n, d, h, self.weights, self.y,
                                          self.fwd_ws, self.status, stream)
        _lib.moe_unpermute_combine(self.y, self.inv_map, weights, T, k, d, self.out, stream)
        return self.out
