"""AdamW reads where its tensors lie at every step: parameters and copies that an assignment to .data has moved are checked again,
for what the kernel takes their sizes and types to be and for overlaps. Without a GPU on stand-ins for CUDA tensors, which
the checks see before anything is written."""
import ctypes

import pytest
import torch

from ragged_grouped_gemm_device_gb300 import _lib, optim


class Fake:
    def __init__(self, at, n, dtype=torch.float32, device=0, contiguous=True):
        self.at, self.n, self.dtype, self.device, self.dense, self.is_cuda = at, n, dtype, device, contiguous, True

    def is_contiguous(self):
        return self.dense

    def get_device(self):
        return self.device

    def numel(self):
        return self.n

    def element_size(self):
        return 2 if self.dtype == torch.bfloat16 else 4

    def data_ptr(self):
        return self.at


def _table(params, copies):
    t = (_lib.AdamWTensor * len(params))()
    for q, p, c in zip(t, params, copies):
        q.n, q.p_dtype, q.p, q.copy = p.n, _lib.DTYPE_BF16 if p.dtype == torch.bfloat16 else _lib.DTYPE_F32, p.at, c and c.at
    return t


BF = torch.bfloat16


@pytest.mark.parametrize("what,bad", [("copies", [Fake(9000, 5, BF), None]), ("copies", [Fake(9000, 10), None]), ("copies", [Fake(9000, 10, BF, 1), None]),
                                      ("copies", [Fake(9000, 10, BF, contiguous=False), None]), ("copies", [Fake(1036, 10, BF), None]),
                                      ("params", [Fake(1000, 10), Fake(1032, 8)]), ("params", [Fake(8998, 10), Fake(2000, 8)])])
def test_what_has_moved_is_checked(what, bad):
    good = dict(params=[Fake(1000, 10), Fake(2000, 8)], copies=[Fake(9000, 10, BF), None])
    t = _table(**good)
    before = bytes(t)
    with pytest.raises(ValueError):
        optim._pointers(t, 0, grads=[Fake(4000, 10), Fake(5000, 8)], **{**good, what: bad})
    assert bytes(t) == before and ctypes.sizeof(t) == 160


@pytest.mark.gpu
@pytest.mark.parametrize("compiled", [False, True])
def test_steps_after_a_move(lib, compiled, monkeypatch):
    if not compiled:
        monkeypatch.setattr(_lib, "adamw_pointers", None)
    elif _lib.adamw_pointers is None:
        pytest.skip("the extension is not built")
    pool = torch.zeros(64, device="cuda")
    p, q, c = torch.ones(10, device="cuda"), torch.ones(8, device="cuda"), torch.zeros(10, dtype=BF, device="cuda")
    opt = optim.AdamW([p, q], copies=[c, None], lr=1e-2)
    grads = [torch.ones_like(p), torch.ones_like(q)]
    opt.step(grads)
    keep = [t.data for t in (p, q, c)]
    for moves in ([(p, pool[:10]), (q, pool[5:13])], [(p, pool[:10]), (c, pool.view(BF)[10:20])], [(c, c.data[:5])], [(c, c.data.float())],
                  [(q, p.data[2:])]):
        for t, to in moves:
            t.data = to
        with pytest.raises(ValueError):
            opt.step(grads)
        for t, to in zip((p, q, c), keep):
            t.data = to
    assert opt.steps == 1 and (pool == 0).all()
    # moved apart: the step goes there
    p.data, c.data = pool[:10].copy_(p.data), pool.view(BF)[100:110]
    opt.step(grads)
    assert opt.steps == 2 and torch.equal(c, p.bfloat16()) and pool[:10].max() < 1.0 - 1e-2 and (pool[10:50] == 0).all()
    opt.step(grads)
    assert opt.steps == 3
