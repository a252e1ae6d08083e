"""A pre-norm mixture-of-experts block on the library's calls:

    n = layer_norm(x);  logits = n W_router^T;  ids, weights = gate(logits)
    out = x + sum_j weights[:, j] expert[ids[:, j]](n)

with the balance and z losses of the gate, and the gradient of all of it. The experts are an
ExpertLayer (BF16: training and serving) or an Mxfp4ExpertLayer (4-bit: serving). The router's
projection and its gradients are torch products in fp32 (TF32 where torch is set to it), the residual
additions torch additions; every other step is a library kernel. Rows are bf16 between the steps: out is
the rounded sum of x and the rounded expert rows; in the backward the experts' gradient of n is rounded,
then its sum with the router's, then the layer norm's dx, then dx + dout. Buffers are allocated once per shape and reused, so what forward() and
backward() return is overwritten by the next call. The calls record no autograd history (what they return
requires no gradient); the gradients are backward()'s.
"""
from __future__ import annotations

import torch

from . import _lib
from .layer import ExpertLayer, _dense


def _version(t: torch.Tensor):
    """The count of in-place changes that torch keeps of a tensor (None for an inference tensor, which has none)."""
    return None if t.is_inference() else t._version


class MoEBlock:
    """gamma, beta [d] (fp32 or bf16), w_router [E, d] fp32, experts over E experts of width d."""

    def __init__(self, gamma: torch.Tensor, beta: torch.Tensor, w_router: torch.Tensor, experts, top_k: int,
                 renorm: bool = True, eps: float = 1e-5):
        E, d = w_router.shape
        assert w_router.dtype == torch.float32 and (E, d) == (experts.E, experts.d)
        assert gamma.shape == (d,) and beta.shape == (d,) and 1 <= top_k <= min(E, 32)
        # as given, views too: a dense copy made here would not follow an optimizer's updates
        self.gamma, self.beta, self.w_router = gamma, beta, w_router
        self.experts, self.E, self.d, self.k, self.eps = experts, E, d, top_k, eps
        self.flags = _lib.GATE_RENORM if renorm else 0
        self.device = w_router.device
        self._T = None

    def _buffers(self, T: int):
        if self._T == T:
            return
        f32, i32, bf = torch.float32, torch.int32, torch.bfloat16
        E, d, k = self.E, self.d, self.k
        new = lambda *shape, dtype=f32: torch.empty(*shape, dtype=dtype, device=self.device)  # noqa: E731
        room = lambda *a: new(max(1, _lib.moe_workspace_bytes(*a)), dtype=torch.uint8)  # noqa: E731
        self.normed, self.mean, self.rstd = new(T, d, dtype=bf), new(T), new(T)
        self.logits, self.ids, self.weights, self.lse = new(T, E), new(T, k, dtype=i32), new(T, k), new(T)
        self.counts, self.n_valid, self.prob_sum, self.loss = new(E, dtype=i32), new(1, dtype=i32), new(E), new(2)
        self.gate_ws, self.norm_ws = room(_lib.OP_GATE, T, k, E), room(_lib.OP_LAYER_NORM_BWD, T, 1, 1, d)
        self.dlogits, self.dnormed, self.dx = new(T, E), new(T, d, dtype=bf), new(T, d, dtype=bf)
        self.dgamma, self.dbeta = new(d), new(d)
        self._T = T

    @torch.no_grad()
    def forward(self, x: torch.Tensor, token_mask: torch.Tensor = None) -> torch.Tensor:
        """x [T, d] bf16 (any row pitch) -> out [T, d] bf16. token_mask nullable [T] bool: padding tokens
        (False) are routed nowhere, count in no loss and pass through the residual unchanged. `loss`
        holds the balance and the z loss, `counts` the slots per expert. x, gamma and w_router are not copied:
        backward() reads them again and refuses when one was changed in place since."""
        if x.dim() != 2 or x.shape[1] != self.d or x.dtype != torch.bfloat16 or x.device != self.device:
            raise ValueError(f"x has to be [T, {self.d}] bfloat16 on {self.device}")
        T = x.shape[0]
        if token_mask is not None and tuple(token_mask.shape) != (T,):
            raise ValueError(f"token_mask has to be [{T}]")
        self._buffers(T)
        self.x = x  # read again by backward(), like gamma and w_router
        self._read = [(t, _version(t)) for t in (x, self.gamma, self.w_router)]
        _lib.moe_layer_norm_fwd(x, _dense(self.gamma), _dense(self.beta), T, self.d, self.eps, self.normed, self.mean, self.rstd)
        torch.mm(self.normed.float(), self.w_router.t(), out=self.logits)
        _lib.moe_gate_fwd(self.logits, token_mask, T, self.k, self.E, self.flags, self.ids, self.weights, self.lse,
                          self.counts, self.n_valid, self.prob_sum, self.loss, self.gate_ws)
        return x + self.experts.forward(self.normed, self.ids, self.weights)

    @torch.no_grad()
    def backward(self, dout: torch.Tensor, d_loss: torch.Tensor = None) -> dict:
        """dout [T, d] bf16, d_loss nullable [2] fp32 (the gradients of the two losses) -> the gradients
        dx (bf16), gamma, beta, w_router, w_ug, w_down (fp32) of the last forward."""
        if not isinstance(self.experts, ExpertLayer):
            raise TypeError("4-bit experts have no backward: train on an ExpertLayer")
        if any(_version(t) != v for t, v in self._read):
            raise RuntimeError("x, gamma or w_router was changed in place since forward(): their gradients would be wrong")
        T = self._T
        if tuple(dout.shape) != (T, self.d) or dout.dtype != torch.bfloat16 or dout.device != self.device:
            raise ValueError(f"dout has to be [{T}, {self.d}] bfloat16 on {self.device}")
        dout = _dense(dout)
        dn, dw_ug, dw_down, dweights = self.experts.backward(dout)
        _lib.moe_gate_bwd(self.logits, self.lse, self.ids, self.weights, self.counts, self.n_valid, dweights, d_loss, T,
                          self.k, self.E, self.flags, self.dlogits)
        dw_router = torch.mm(self.dlogits.t(), self.normed.float())
        self.dnormed.copy_(torch.addmm(dn.float(), self.dlogits, self.w_router))
        _lib.moe_layer_norm_bwd(self.dnormed, self.x, _dense(self.gamma), self.mean, self.rstd, T, self.d, self.dx, self.dgamma,
                                self.dbeta, self.norm_ws)
        return dict(dx=self.dx + dout, gamma=self.dgamma, beta=self.dbeta, w_router=dw_router, w_ug=dw_ug, w_down=dw_down)
