"""AdamW over all tensors of a model in one launch, on the library's calls.

    opt = AdamW(list(block.tensors().values()), lr=3e-4, weight_decay=0.1, state_bits=8, max_norm=1.0)
    grads = block.backward(dout, d_loss)
    norm = opt.step([grads[name] for name in block.tensors()])

States are fp32, or 8 bits (E4M3 elements in blocks of 32 with a power-of-two scale, of m and of sqrt(v), rounded
stochastically). A parameter is fp32, optionally with a bf16 copy that the step refreshes (a master weight and the
weight that the products read), or bf16 alone, rounded stochastically. step() allocates nothing and can be captured
in a CUDA graph: the step count, the gradients' norm and a learning rate's factor stay on the device.
"""
from __future__ import annotations

import torch

from . import _lib

BLOCK = 32  # elements of a scale of the 8-bit states


def _dense(t, device, what):
    if not t.is_cuda or not t.is_contiguous() or t.get_device() != device or t.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"{what} has to be a dense bfloat16 or float32 tensor on cuda:{device}")


def _apart(tensors):
    """A step would update elements that two tensors share twice."""
    spans = sorted((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in tensors if t is not None and t.numel())
    if any(a[1] > b[0] for a, b in zip(spans, spans[1:])):
        raise ValueError("parameters and copies may not overlap: a step would update the shared elements twice")


def _pointers(table, device, params, copies, grads):
    """Write where a step's tensors lie into the table (at every step: an assignment to .data moves a parameter or a copy) and count
    their versions up. What has moved is checked like what the constructor was given. The extension's adamw_pointers does the
    same."""
    moved = False
    for q, p, c, g in zip(table, params, copies, grads):
        _dense(g, device, "a gradient")
        if g.numel() != q.n:
            raise ValueError(f"a gradient has {g.numel()} elements, its parameter {q.n}")
        _dense(p, device, "a parameter")
        if p.numel() != q.n or _lib._dtype(p) != q.p_dtype:
            raise ValueError("a parameter's size or type has changed")
        if c is not None:
            _dense(c, device, "a copy")
            if c.numel() != q.n or c.dtype != torch.bfloat16:
                raise ValueError("a copy's size or type has changed")
        moved |= p.data_ptr() != (q.p or 0) or (0 if c is None else c.data_ptr()) != (q.copy or 0)
    if moved:
        _apart((*params, *copies))
    for q, p, c, g in zip(table, params, copies, grads):
        q.g, q.g_dtype, q.p, q.copy = g.data_ptr(), _lib._dtype(g), p.data_ptr(), None if c is None else c.data_ptr()
    torch.autograd.graph.increment_version([t for t in (*params, *copies) if t is not None and not t.is_inference()])


class AdamW:
    """params: dense CUDA tensors of one device, bf16 or fp32, updated in place. weight_decay: one number, or one for each
    parameter. copies: for each parameter None or a bf16 tensor of its shape (fp32 parameters only). max_norm: the
    gradients are scaled so that their global norm is at most this; where it is not finite the step is skipped.
    lr_scale: nullable fp32 [1] on the device, a factor of lr that is read when the step runs.

    `m`, `v` (and `m_scale`, `v_scale` of 8-bit states) are flat buffers in which parameter i has the elements
    starts[i] to starts[i] + numel, starts[i] a multiple of 32; they and `steps` are what a checkpoint keeps and what is
    copied back into them. What lies between two parameters stays 0."""

    def __init__(self, params, lr: float = 1e-3, betas=(0.9, 0.999), eps: float = 1e-8, weight_decay=0.01,
                 state_bits: int = 32, copies=None, max_norm: float = None, seed: int = 0, lr_scale: torch.Tensor = None):
        params = list(params)
        if not params:
            raise ValueError("there are no parameters")
        if state_bits not in (32, 8):
            raise ValueError("state_bits has to be 32 or 8")
        decays = list(weight_decay) if isinstance(weight_decay, (list, tuple)) else [weight_decay] * len(params)
        copies = [None] * len(params) if copies is None else list(copies)
        if len(decays) != len(params) or len(copies) != len(params):
            raise ValueError("weight_decay and copies have to have one entry for each parameter")
        self.device = params[0].device
        for p, c in zip(params, copies):
            _dense(p, self.device.index, "a parameter")
            if c is not None and (c.dtype != torch.bfloat16 or c.shape != p.shape or p.dtype != torch.float32):
                raise ValueError("a copy has to be bfloat16, of the shape of its float32 parameter")
            if c is not None:
                _dense(c, self.device.index, "a copy")
        _apart((*params, *copies))
        if max_norm is not None and not 0 < max_norm < float("inf"):
            raise ValueError("max_norm has to be positive and finite")
        self.params, self.copies, self.state_bits = params, copies, state_bits
        self.lr, self.betas, self.eps, self.max_norm, self.seed = lr, tuple(betas), eps, max_norm, seed
        if lr_scale is not None and lr_scale.device != self.device:
            raise ValueError(f"lr_scale has to be on {self.device}")
        self.lr_scale = lr_scale
        self.starts, total = [], 0
        for p in params:
            self.starts.append(total)
            total += (p.numel() + BLOCK - 1) // BLOCK * BLOCK
        new = lambda n, dtype: torch.zeros(n, dtype=dtype, device=self.device)  # noqa: E731
        kind = torch.float32 if state_bits == 32 else torch.uint8
        self.m, self.v = new(total, kind), new(total, kind)
        self.m_scale, self.v_scale = (new(total // BLOCK, torch.uint8) if state_bits == 8 else None for _ in range(2))
        self._steps, self._norm = new(2, torch.int32), new(2, torch.float32)
        self._ws = new(max(1, _lib.moe_workspace_bytes(_lib.OP_GRAD_NORM, 0, 1, 1)), torch.uint8)
        self._table = (_lib.AdamWTensor * len(params))()
        size = self.m.element_size()
        for q, p, c, at, decay in zip(self._table, params, copies, self.starts, decays):
            q.n, q.weight_decay, q.p_dtype = p.numel(), decay, _lib._dtype(p)
            q.m, q.v = self.m.data_ptr() + at * size, self.v.data_ptr() + at * size
            if state_bits == 8:
                q.m_scale, q.v_scale = self.m_scale.data_ptr() + at // BLOCK, self.v_scale.data_ptr() + at // BLOCK

    @property
    def steps(self) -> int:
        """Steps done (reads the device)."""
        return int(self._steps[0].item())

    @steps.setter
    def steps(self, n: int):
        self._steps[0] = n

    @torch.no_grad()
    def step(self, grads, stream=None):
        """One step with a gradient (bf16 or fp32, of the parameter's size) for each parameter. Returns the gradients' global norm
        (a tensor of no dimension that the next step overwrites), or None without max_norm."""
        if len(grads) != len(self.params):
            raise ValueError(f"expected {len(self.params)} gradients, not {len(grads)}")
        _lib.load()
        (_lib.adamw_pointers or _pointers)(self._table, self.device.index, self.params, self.copies, grads)
        scale = None
        if self.max_norm is not None:
            _lib.moe_grad_norm(self._table, self.max_norm, self._norm, self._ws, stream)
            scale = self._norm[1:]
        _lib.moe_adamw_step(self._table, self.state_bits, self.lr, *self.betas, self.eps, self.seed, self._steps,
                            self.lr_scale, scale, stream)
        return None if scale is None else self._norm[0]
