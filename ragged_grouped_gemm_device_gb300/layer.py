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


def _hold_captured(owner):
    """Called wherever `owner` is about to use its buffers: while a graph is captured they are kept as long as owner lives, because
    calls of other sizes put others in their place and the graph goes on to use these."""
    if torch.cuda.is_current_stream_capturing():
        owner.__dict__.setdefault("_captured", []).append([t for t in vars(owner).values() if isinstance(t, torch.Tensor)])


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
        self.runs = 0  # forwards begun: each one overwrites what the backward of the one before reads
        self.status = torch.zeros(1, dtype=torch.int32, device=self.device)

    def _buffers(self, T: int, k: int):
        if self._key != (T, k):
            self._allocate(T, k)
        _hold_captured(self)

    def _allocate(self, T: int, k: int):
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
        self.runs += 1
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
        if self._key != (T, k):
            self._allocate(T, k)
        _hold_captured(self)

    def _allocate(self, T: int, k: int):
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


class Int4ExpertLayer:
    """The forward of one SwiGLU expert layer on 4-bit integer weights with group scales and bf16 activations, for few
    tokens (decoding; no backward).

    Takes the bf16 weights of ExpertLayer and quantizes them once (the bf16 tensors are not kept), or, through
    from_checkpoint, codes, scales and zero points. Any d and h. More than 4096 token slots run in pieces that
    each read the weights: long prompts are Mxfp4ExpertLayer's and ExpertLayer's."""

    def __init__(self, w_ug: torch.Tensor, w_down: torch.Tensor, group: int = 128, stream=None):
        E, two_h, d = w_ug.shape
        h = two_h // 2
        assert w_down.shape == (E, h, d) and two_h == 2 * h
        assert w_ug.dtype == torch.bfloat16 and w_down.dtype == torch.bfloat16
        with _on(stream):
            # contractions along d and along h: rows of W_down^T
            parts = [self._quantize(w, group, stream) for w in (_dense(w_ug), w_down.transpose(1, 2).contiguous())]
        self._pack(E, d, h, group, parts, stream)

    @classmethod
    def from_checkpoint(cls, ug, down, E: int, d: int, h: int, group: int, stream=None):
        """ug, down: (codes uint8 [..., ceil(K / 2)], scales bf16 [..., groups], zeros uint8 [..., groups] or None) of
        W_ug [E, 2h, d] along d and of W_down^T [E, d, h] along h."""
        self = cls.__new__(cls)
        with _on(stream):
            parts = [tuple(None if t is None else _dense(t) for t in part) for part in (ug, down)]
        self._pack(E, d, h, group, parts, stream)
        return self

    @staticmethod
    def _quantize(w, group, stream):
        K, rows, dev = w.shape[-1], w.numel() // w.shape[-1], w.device
        groups = (K + group - 1) // group
        codes = torch.empty(rows, (K + 1) // 2, dtype=torch.uint8, device=dev)
        scales = torch.empty(rows, groups, dtype=torch.bfloat16, device=dev)
        zeros = torch.empty(rows, groups, dtype=torch.uint8, device=dev)
        _lib.moe_w4_quantize_rows(w, rows, K, group, codes, scales, zeros, stream)
        return codes, scales, zeros

    def _pack(self, E, d, h, group, parts, stream):
        self.E, self.d, self.h, self.group = E, d, h, group
        self.device = parts[0][0].device
        packed = []
        with _on(stream):
            for (codes, scales, zeros), (matrices, N, K) in zip(parts, ((2 * E, h, d), (E, d, h))):
                n = _lib.moe_workspace_bytes(_lib.OP_W4_WEIGHTS, 0, 1, matrices, K, N, group)
                w = torch.empty(max(n, 1), dtype=torch.uint8, device=self.device)
                _lib.moe_w4_pack(codes, scales, zeros, matrices, N, K, group, w, stream)
                packed.append(w)
        self.w_ug, self.w_down = packed
        self._key = None

    def _buffers(self, T: int, k: int):
        if self._key != (T, k):
            self._allocate(T, k)
        _hold_captured(self)

    def _allocate(self, T: int, k: int):
        piece = min(T, _lib.W4_MAX_SLOTS // k)
        n = _lib.moe_workspace_bytes(_lib.OP_W4_DECODE, piece, k, self.E, self.d, self.h)
        self.ws = torch.empty(max(n, 1), dtype=torch.uint8, device=self.device)
        self.out = torch.empty(T, self.d, dtype=torch.bfloat16, device=self.device)
        self._key = (T, k)

    def forward(self, x: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, stream=None):
        """x [T, d] bf16 (any row pitch), ids [T, k] int32, weights [T, k] fp32 -> out [T, d] bf16."""
        if ids.dim() != 2 or ids.dtype != torch.int32:
            raise ValueError("ids has to be [T, k] int32")
        T, k = ids.shape
        if not 1 <= k <= 32:
            raise ValueError("k has to be 1 to 32")
        if tuple(x.shape) != (T, self.d) or x.dtype != torch.bfloat16:
            raise ValueError(f"x has to be [{T}, {self.d}] bfloat16")
        if tuple(weights.shape) != (T, k) or weights.dtype != torch.float32:
            raise ValueError(f"weights has to be [{T}, {k}] float32")
        with _on(stream):
            ids, weights = _dense(ids), _dense(weights)
            x = x if x.stride(1) == 1 else _dense(x)
            self._buffers(T, k)
        piece = _lib.W4_MAX_SLOTS // k
        for t in range(0, T, piece):
            n = min(piece, T - t)
            _lib.moe_w4_swiglu_decode(x[t:t + n], ids[t:t + n], weights[t:t + n], n, k, self.E, self.d, self.h, self.group,
                                      self.w_ug, self.w_down, self.out[t:t + n], self.ws, stream)
        return self.out
