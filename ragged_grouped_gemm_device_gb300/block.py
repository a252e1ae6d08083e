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

A block may have another kind of norm in front, a norm behind it, a gate for each channel and scales:

    n = pre(x);  y = sum_j weights[:, j] expert[ids[:, j]](n);  out = res_scale x + branch_scale gate post(y)

and a MoEStack runs several such blocks, the join behind one and the norm in front of the next in one pass. There the
residual additions are in fp32 and rounded once.
"""
from __future__ import annotations

import torch

from . import _lib
from .layer import ExpertLayer, _dense, _hold_captured

_ITSELF = "itself"  # who asked for a plain block's last run

_NORMS = {"none": _lib.NORM_NONE, "layer": _lib.NORM_LAYER, "rms": _lib.NORM_RMS}


def _version(t: torch.Tensor):
    """The count of in-place changes that torch keeps of a tensor (None for an inference tensor, which has none)."""
    return None if t.is_inference() else t._version


class MoEBlock:
    """gamma, beta [d] (fp32 or bf16; beta None with an RMS norm), w_router [E, d] fp32, experts over E experts of width d.
    pre: "layer" or "rms"; post: "none", "layer" or "rms", with post_gamma and post_beta [d] (each nullable); gate
    nullable [d]. All norm weights and the gate are of one type."""

    def __init__(self, gamma: torch.Tensor, beta: torch.Tensor, w_router: torch.Tensor, experts, top_k: int,
                 renorm: bool = True, eps: float = 1e-5, *, pre: str = "layer", post: str = "none",
                 post_gamma: torch.Tensor = None, post_beta: torch.Tensor = None, gate: torch.Tensor = None,
                 res_scale: float = 1.0, branch_scale: float = 1.0):
        E, d = w_router.shape
        assert w_router.dtype == torch.float32 and (E, d) == (experts.E, experts.d)
        assert gamma.shape == (d,) and 1 <= top_k <= min(E, 32)
        assert pre in ("layer", "rms") and post in _NORMS
        assert (beta is None) if pre == "rms" else beta.shape == (d,)
        assert post != "none" or post_gamma is None
        assert post == "layer" or post_beta is None
        assert all(t is None or t.shape == (d,) for t in (post_gamma, post_beta, gate))
        # as given, views too: a dense copy made here would not follow an optimizer's updates
        self.gamma, self.beta, self.w_router = gamma, beta, w_router
        self.post_gamma, self.post_beta, self.gate = post_gamma, post_beta, gate
        self.pre, self.post, self.res_scale, self.branch_scale = pre, post, res_scale, branch_scale
        self.plain = pre == "layer" and post == "none" and gate is None and res_scale == 1.0 and branch_scale == 1.0
        self.experts, self.E, self.d, self.k, self.eps = experts, E, d, top_k, eps
        self.flags = _lib.GATE_RENORM if renorm else 0
        self.device = w_router.device
        self._T = self._ran = None
        self._joins = None if self.plain else _Joins()

    def _buffers(self, T: int):
        if self._T != T:
            self._allocate(T)
        _hold_captured(self)

    def _allocate(self, T: int):
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
        (False) are routed nowhere and count in no loss; their y is a row of zeros, and out is what the formula makes of
        it: x, with scales and a norm behind the block res_scale x + branch_scale gate post(0), where a layer norm's post(0)
        is post_beta. They have a share in the gradients of post_beta and of the gate there unless dout is 0 in their rows. `loss`
        holds the balance and the z loss, `counts` the slots per expert. x and the weights, the experts' among them, are not
        copied: backward() reads them again and refuses when one was changed in place since."""
        if not self.plain:
            return self._joins.forward([self], x, token_mask)
        T = self._check(x, token_mask)
        self._buffers(T)
        self._ran = None  # until all of it has run: a call that raises leaves buffers of two runs
        self.x = x  # read again by backward(), like the weights
        self._read = [(t, _version(t)) for t in (x, *self.tensors().values())]
        _lib.moe_layer_norm_fwd(x, _dense(self.gamma), _dense(self.beta), T, self.d, self.eps, self.normed, self.mean, self.rstd)
        out = x + self._route(token_mask)
        self._ran = _ITSELF
        return out

    def _check(self, x, token_mask) -> int:
        if x.dim() != 2 or x.shape[1] != self.d or x.dtype != torch.bfloat16 or x.device != self.device:
            raise ValueError(f"x has to be [T, {self.d}] bfloat16 on {self.device}")
        if token_mask is not None and tuple(token_mask.shape) != (x.shape[0],):
            raise ValueError(f"token_mask has to be [{x.shape[0]}]")
        return x.shape[0]

    def _route(self, token_mask):
        """The experts' combined rows of self.normed."""
        T = self._T
        torch.mm(self.normed.float(), self.w_router.t(), out=self.logits)
        _lib.moe_gate_fwd(self.logits, token_mask, T, self.k, self.E, self.flags, self.ids, self.weights, self.lse,
                          self.counts, self.n_valid, self.prob_sum, self.loss, self.gate_ws)
        y = self.experts.forward(self.normed, self.ids, self.weights)
        self._experts_run = getattr(self.experts, "runs", None)
        return y

    def _route_backward(self, dy, d_loss) -> dict:
        """The gradient of self.normed, left in self.dnormed, and those of the router's and the experts' weights."""
        dn, dw_ug, dw_down, dweights = self.experts.backward(dy)
        _lib.moe_gate_bwd(self.logits, self.lse, self.ids, self.weights, self.counts, self.n_valid, dweights, d_loss, self._T,
                          self.k, self.E, self.flags, self.dlogits)
        dw_router = torch.mm(self.dlogits.t(), self.normed.float())
        self.dnormed.copy_(torch.addmm(dn.float(), self.dlogits, self.w_router))
        return dict(w_router=dw_router, w_ug=dw_ug, w_down=dw_down)

    @torch.no_grad()
    def backward(self, dout: torch.Tensor, d_loss: torch.Tensor = None) -> dict:
        """dout [T, d] bf16, d_loss nullable [2] fp32 (the gradients of the two losses) -> the gradients
        dx (bf16), gamma, beta, w_router, w_ug, w_down (fp32) of the last forward."""
        if not self.plain:
            grads = self._joins.backward([self], dout, None if d_loss is None else [d_loss])
            return dict(dx=grads["dx"], **grads["blocks"][0])
        self._check_backward(dout, _ITSELF)
        T = self._T
        dout = _dense(dout)
        grads = self._route_backward(dout, d_loss)
        _lib.moe_layer_norm_bwd(self.dnormed, self.x, _dense(self.gamma), self.mean, self.rstd, T, self.d, self.dx, self.dgamma,
                                self.dbeta, self.norm_ws)
        return dict(dx=self.dx + dout, gamma=self.dgamma, beta=self.dbeta, **grads)

    def _check_backward(self, dout, owner):
        if not isinstance(self.experts, ExpertLayer):
            raise TypeError("4-bit experts have no backward: train on an ExpertLayer")
        if self._ran is not owner:
            raise RuntimeError("the block's buffers hold no whole run of this model: another one followed, or its forward() raised")
        if self._experts_run != self.experts.runs:
            raise RuntimeError("the experts' buffers hold another run: their forward() was called by itself or by another block")
        if any(_version(t) != v for t, v in self._read):
            raise RuntimeError("x or a weight was changed in place since forward(): the gradients would be wrong")
        if tuple(dout.shape) != (self._T, self.d) or dout.dtype != torch.bfloat16 or dout.device != self.device:
            raise ValueError(f"dout has to be [{self._T}, {self.d}] bfloat16 on {self.device}")

    def tensors(self) -> dict:
        """The block's trained tensors, by the names of their gradients."""
        every = dict(gamma=self.gamma, beta=self.beta, post_gamma=self.post_gamma, post_beta=self.post_beta, gate=self.gate,
                     w_router=self.w_router)
        if isinstance(self.experts, ExpertLayer):
            every.update(w_ug=self.experts.w_ug, w_down=self.experts.w_down)
        return {n: t for n, t in every.items() if t is not None}


class _Joins:
    """The joins of a run through blocks, and their buffers. It holds no block, whose memory would wait for the garbage
    collector if the block held it."""

    def __init__(self):
        self._T = None

    def _buffers(self, blocks, T: int):
        for b in blocks:
            b._buffers(T)
        if self._T != T:
            self._allocate(blocks, T)
        _hold_captured(self)

    def _allocate(self, blocks, T: int):
        d, dev, count = blocks[0].d, blocks[0].device, len(blocks)
        new = lambda *shape, dtype=torch.float32: torch.empty(*shape, dtype=dtype, device=dev)  # noqa: E731
        self.rows = new(count, T, d, dtype=torch.bfloat16)       # r behind each block
        self.stats = new(count + 1, 4, T)                        # of join i, the one in front of block i
        self.dx, self.dy = new(T, d, dtype=torch.bfloat16), new(T, d, dtype=torch.bfloat16)
        self.ws = new(max(1, _lib.moe_workspace_bytes(_lib.OP_RESIDUAL_NORM_BWD, T, 1, 1, d)), dtype=torch.uint8)
        self._T = T

    @staticmethod
    def _join(blocks, i):
        """The weights of join i, between blocks i - 1 and i: (post, gamma, beta, gate, pre, gamma, beta), then eps and scales."""
        behind = blocks[i - 1] if i > 0 else None
        ahead = blocks[i] if i < len(blocks) else None
        dense = lambda b, n: None if b is None or getattr(b, n) is None else _dense(getattr(b, n))  # noqa: E731
        weights = (_NORMS[behind.post] if behind else _lib.NORM_NONE, dense(behind, "post_gamma"), dense(behind, "post_beta"),
                   dense(behind, "gate"), _NORMS[ahead.pre] if ahead else _lib.NORM_NONE, dense(ahead, "gamma"), dense(ahead, "beta"))
        return weights, (ahead or behind).eps, (behind.res_scale, behind.branch_scale) if behind else (1.0, 1.0)

    @torch.no_grad()
    def forward(self, blocks, x: torch.Tensor, token_mask: torch.Tensor) -> torch.Tensor:
        T, d = blocks[0]._check(x, token_mask), blocks[0].d
        self._buffers(blocks, T)
        for b in blocks:
            b._ran = None
        if x.untyped_storage().data_ptr() == self.rows.untyped_storage().data_ptr():
            x = x.clone()  # an earlier output: this forward writes there, and backward() reads x again
        r, y = x, None
        self._ys = []
        for i in range(len(blocks) + 1):
            weights, eps, scales = self._join(blocks, i)
            n = blocks[i].normed if i < len(blocks) else None
            to = self.rows[i - 1] if i > 0 else None
            _lib.moe_residual_norm_fwd(r, y, *weights, T, d, eps, *scales, to, n, self.stats[i])
            if i > 0:
                r = to
            if n is not None:
                y = blocks[i]._route(token_mask)
                self._ys.append(y)
        self.x = x
        for b in blocks:
            b._read = [(t, _version(t)) for t in b.tensors().values()]
            b._ran = self
        blocks[0]._read.append((x, _version(x)))
        if not self.rows.is_inference():  # whoever holds an earlier output for a backward learns that it has changed
            torch.autograd.graph.increment_version(self.rows)
        return r

    @torch.no_grad()
    def backward(self, blocks, dout: torch.Tensor, d_loss) -> dict:
        if self._T is None:
            raise RuntimeError("backward() before forward()")
        for b in blocks:
            b._check_backward(dout, self)
        count, T, d = len(blocks), self._T, blocks[0].d
        losses = [None] * count if d_loss is None else list(d_loss)
        if len(losses) != count:
            raise ValueError("d_loss has to have one entry for each block")
        grads = [{} for _ in blocks]
        new = lambda: torch.empty(d, dtype=torch.float32, device=dout.device)  # noqa: E731
        dr, dn = _dense(dout), None
        for i in range(count, -1, -1):
            weights, _, scales = self._join(blocks, i)
            out = [None] * 5   # d_post_gamma, d_post_beta, d_gate, d_pre_gamma, d_pre_beta
            for j, (w, owner, name) in enumerate(zip(weights[1:4] + weights[5:], (i - 1,) * 3 + (i,) * 2,
                                                     ("post_gamma", "post_beta", "gate", "gamma", "beta"))):
                if w is not None:
                    out[j] = grads[owner][name] = new()
            r = None if dn is None else self.rows[i - 1] if i > 0 else self.x
            y, dy = (self._ys[i - 1], self.dy) if i > 0 else (None, None)
            _lib.moe_residual_norm_bwd(dn, dr, r, y, *weights[:5], weights[5], self.stats[i], T, d, *scales, self.dx, dy,
                                       *out, self.ws)
            dr = self.dx
            if i > 0:
                grads[i - 1].update(blocks[i - 1]._route_backward(self.dy, losses[i - 1]))
                dn = blocks[i - 1].dnormed
        return dict(dx=self.dx, blocks=grads)


class MoEStack:
    """Blocks of one width, one behind the other: the norm behind a block, its gate and scales, the residual addition and the
    norm in front of the next block are one call. Every block has experts of its own."""

    def __init__(self, blocks):
        self.blocks = list(blocks)
        if not self.blocks:
            raise ValueError("there are no blocks")
        first = self.blocks[0]
        if any((b.d, b.device) != (first.d, first.device) for b in self.blocks):
            raise ValueError("the blocks have to be of one width and on one device")
        if len({id(b.experts) for b in self.blocks}) < len(self.blocks) or len({id(b) for b in self.blocks}) < len(self.blocks):
            raise ValueError("every block has to have experts of its own: their buffers hold what the backward reads")
        # a join has one eps for the norms on both its sides
        if any(a.post != "none" and a.eps != b.eps for a, b in zip(self.blocks, self.blocks[1:])):
            raise ValueError("a block with a norm behind it has to have the eps of the next block")
        self.d, self._joins = first.d, _Joins()

    def forward(self, x: torch.Tensor, token_mask: torch.Tensor = None) -> torch.Tensor:
        """x [T, d] bf16 (any row pitch) -> out [T, d] bf16, a buffer that the next forward overwrites. token_mask as in
        MoEBlock.forward: a padding token's rows take part in no block's experts or losses, but in its joins. The blocks hold
        their losses and counts. x and the weights are not copied: backward() reads them again and refuses when one was changed
        in place since."""
        return self._joins.forward(self.blocks, x, token_mask)

    def backward(self, dout: torch.Tensor, d_loss=None) -> dict:
        """dout [T, d] bf16, d_loss: None or for each block None or [2] fp32 -> dx (bf16) and blocks, a list of each
        block's gradients by the names of its tensors(); dx is a buffer that the next backward overwrites."""
        return self._joins.backward(self.blocks, dout, d_loss)
