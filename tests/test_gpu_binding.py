"""The compiled binding against the Python functions that it replaces: the same results from the same
arguments (positional or by keyword), the same kinds of refusal."""
import inspect

import pytest
import torch

from ragged_grouped_gemm_device_gb300 import _lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def both(lib):
    from ragged_grouped_gemm_device_gb300 import _binding  # built next to the library
    assert set(_lib.PYTHON_BINDING) == set(_lib.COMPILED)
    assert all(getattr(_lib, n) is getattr(_binding, n) for n in _lib.COMPILED)
    return {n: (_lib.PYTHON_BINDING[n], getattr(_binding, n)) for n in _lib.COMPILED}


def _calls():
    """(name, function of a fresh output filling -> (args by name, outputs)) of every call."""
    T, E, k, d, h = 37, 8, 3, 64, 96
    g = torch.Generator("cuda").manual_seed(3)
    n = lambda *s, dtype=torch.float32: torch.randn(*s, generator=g, device="cuda").to(dtype)
    new = lambda *s, dtype=torch.float32: torch.full(s, 7, dtype=dtype, device="cuda")
    room = lambda *a: torch.zeros(max(1, _lib.moe_workspace_bytes(*a)), dtype=torch.uint8, device="cuda")
    bf, i32, u8 = torch.bfloat16, torch.int32, torch.uint8
    x, dy, gamma, beta = n(T, d + 3, dtype=bf)[:, 1:1 + d], n(T, d, dtype=bf), n(d), n(d)
    mean, rstd = x.float().mean(1), 1 / x.float().std(1)
    logits, mask = n(T, E), torch.rand(T, generator=g, device="cuda") > 0.1
    lse, ids = torch.logsumexp(logits, 1), torch.topk(logits, k).indices.to(i32)
    w, dw, dl = n(T, k), n(T, k), n(2)
    counts = torch.bincount(ids.reshape(-1).long(), minlength=E).to(i32)
    nv = torch.tensor([T], dtype=i32, device="cuda")
    xq, rows = n(T, d, dtype=bf), T * k
    offs = torch.tensor([rows // 2, rows] + [rows] * (E - 2), dtype=i32, device="cuda")
    inv = torch.randperm(rows, generator=g, device="cuda").to(i32)
    mxw = room(_lib.OP_MX4_WEIGHTS, 0, 1, E, d, h)
    _lib.moe_mx4_prepare_weights(n(E, 2 * h, d, dtype=bf), n(E, h, d, dtype=bf), E, d, h, mxw)
    codes, sf = room(_lib.OP_MX4_ROW_SCALES, T, k, E, d, h)[:0].new_zeros(rows, d // 2), room(_lib.OP_MX4_ROW_SCALES, T, k, E, d, h)
    _lib.moe_permute_mxfp4(xq, inv, offs, T, k, E, d, codes, sf)
    yield "moe_layer_norm_fwd", lambda: (dict(x=x, gamma=gamma, beta=beta, T=T, d=d, eps=1e-5, y=(o := new(T, d, dtype=bf)),
                                              mean=(m := new(T)), rstd=(r := new(T))), (o, m, r))
    yield "moe_layer_norm_bwd", lambda: (dict(dy=dy, x=x, gamma=gamma, mean=mean, rstd=rstd, T=T, d=d, dx=(o := new(T, d, dtype=bf)),
                                              dgamma=(p := new(d)), dbeta=(q := new(d)),
                                              ws=room(_lib.OP_LAYER_NORM_BWD, T, 1, 1, d)), (o, p, q))
    yield "moe_gate_fwd", lambda: (dict(logits=logits, token_mask=mask, T=T, top_k=k, E=E, flags=1, ids=(a := new(T, k, dtype=i32)),
                                        weights=(b := new(T, k)), lse=(c := new(T)), counts=(e := new(E, dtype=i32)),
                                        n_valid=(f := new(1, dtype=i32)), prob_sum=(p := new(E)), loss=(q := new(2)),
                                        ws=room(_lib.OP_GATE, T, k, E)), (a, b, c, e, f, p, q))
    yield "moe_gate_bwd", lambda: (dict(logits=logits, lse=lse, ids=ids, weights=w, counts=counts, n_valid=nv, d_weights=dw,
                                        d_loss=dl, T=T, top_k=k, E=E, flags=1, dlogits=(o := new(T, E))), (o,))
    yield "moe_mx4_quantize_rows", lambda: (dict(x=xq, offsets=nv, E=1, cap=T, K=d, q=(o := new(T, d // 2, dtype=u8)),
                                                 sf=(p := room(_lib.OP_MX4_ROW_SCALES, T, 1, 1, d, 32))), (o, p))
    yield "moe_mx4_dequantize_rows", lambda: (dict(q=codes, sf=sf, offsets=offs, E=E, cap=rows, K=d, x=(o := new(rows, d, dtype=bf))), (o,))
    yield "moe_permute_mxfp4", lambda: (dict(x=xq, inv_map=inv, offsets=offs, T=T, top_k=k, E=E, d=d,
                                             q=(o := new(rows, d // 2, dtype=u8)), sf=(p := torch.zeros_like(sf))), (o, p))
    yield "moe_grouped_swiglu_fwd_mxfp4", lambda: (dict(xq=codes, xsf=sf, offsets=offs, E=E, cap=rows, d=d, h=h, mxw=mxw,
                                                        y=(o := new(rows, d, dtype=bf)), ws=room(_lib.OP_MX4_FWD, T, k, E, d, h)), (o,))
    yield "moe_unpermute_combine", lambda: (dict(y=n(rows, d, dtype=bf).fill_(0.5), inv_map=inv, weights=w, T=T, top_k=k, d=d,
                                                 out=(o := new(T, d, dtype=bf))), (o,))
    yield "moe_route_offsets", lambda: (dict(ids=ids, T=T, top_k=k, E=E, counts=(a := new(E, dtype=i32)), offsets=(b := new(E, dtype=i32)),
                                             sorted_src=(c := new(rows, dtype=i32)), inv_map=(e := new(rows, dtype=i32)),
                                             ws=room(_lib.OP_ROUTE, T, k, E)), (a, b, c, e))


def test_same_results_and_refusals(both):
    seen = set()
    for name, make in _calls():
        seen.add(name)
        python, compiled = both[name]
        order = list(inspect.signature(python).parameters)
        results = []
        for fn, positional in ((python, False), (compiled, False), (compiled, True)):
            args, outs = make()
            if positional:
                fn(*[args[p] for p in order if p in args and p not in ("dev_status", "stream")])
            else:
                fn(**args, stream=torch.cuda.current_stream())
            results.append([o.clone() for o in outs])
        for other in results[1:]:
            assert all(torch.equal(a, b) for a, b in zip(results[0], other)), name
        # one argument wrong at a time: the same kind of error from both
        args, _ = make()
        for p, v in args.items():
            wrong = [v.cpu()] if isinstance(v, torch.Tensor) else [-5, "x"]
            if isinstance(v, torch.Tensor) and v.dim() == 2:
                wrong.append(v.t())  # not contiguous
            for bad in wrong:
                kinds = []
                for fn in (python, compiled):
                    try:
                        fn(**{**make()[0], p: bad})
                        kinds.append(None)
                    except Exception as e:  # noqa: BLE001
                        kinds.append(type(e).__name__)
                # a wrong kind of argument: ctypes, a comparison or the conversion to a number may notice it
                kind = {"ArgumentError", "TypeError", "ValueError"}
                assert kinds[0] == kinds[1] or (isinstance(bad, str) and set(kinds) <= kind), (name, p, kinds)
        for fn in (python, compiled):
            with pytest.raises(TypeError):
                fn(**{**args, "nonsense": 1})
            with pytest.raises(TypeError):
                fn()
    assert seen == set(_lib.COMPILED)
