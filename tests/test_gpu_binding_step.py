"""The compiled binding of the residual join, AdamW and the 4-bit integer products against the Python functions that it
replaces: the same results from the same arguments, the same kinds of refusal."""
import inspect

import pytest
import torch

from ragged_grouped_gemm_device_gb300 import _lib, optim

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def both(lib):
    from ragged_grouped_gemm_device_gb300 import _binding  # built next to the library
    assert set(_lib.PYTHON_BINDING_STEP) == set(_lib.COMPILED_STEP)
    assert _lib.adamw_pointers is _binding.adamw_pointers
    return {n: (_lib.PYTHON_BINDING_STEP[n], getattr(_binding, n)) for n in _lib.COMPILED_STEP}


def _table(state):
    t = (_lib.AdamWTensor * 1)()
    p, g, m, v = state
    t[0] = _lib.AdamWTensor(p=p.data_ptr(), g=g.data_ptr(), m=m.data_ptr(), v=v.data_ptr(), n=p.numel(), weight_decay=0.1, p_dtype=1, g_dtype=1)
    return t


def _calls():
    """(name, function of fresh outputs -> (args by name, outputs)) of every call."""
    T, d, E, k, h, group = 19, 72, 5, 3, 40, 32
    g = torch.Generator("cuda").manual_seed(3)
    n = lambda *s, dtype=torch.float32: torch.randn(*s, generator=g, device="cuda").to(dtype)
    new = lambda *s, dtype=torch.float32: torch.full(s, 7, dtype=dtype, device="cuda")
    room = lambda *a: torch.zeros(max(1, _lib.moe_workspace_bytes(*a)), dtype=torch.uint8, device="cuda")
    bf = torch.bfloat16
    x, y, dn, w = n(T, d + 3)[:, 1:1 + d], n(T, d, dtype=bf), n(T, d, dtype=bf), [n(d) for _ in range(5)]
    stats = torch.stack([n(T), 1 + n(T).abs(), n(T), 1 + n(T).abs()])
    yield "moe_residual_norm_fwd", lambda: (dict(x=x, y=y, post=1, post_gamma=w[0], post_beta=w[1], gate=w[2], pre=1, pre_gamma=w[3], pre_beta=w[4],
                                                 T=T, d=d, eps=1e-5, res_scale=0.5, branch_scale=2.0, r=(r := new(T, d)),
                                                 n=(o := new(T, d, dtype=bf)), stats=(s := new(4, T))), (r, o, s))
    yield "moe_residual_norm_bwd", lambda: (dict(dn=dn, dr=x, r=n(T, d).fill_(0.3), y=y, post=1, post_gamma=w[0], post_beta=w[1], gate=w[2], pre=1,
                                                 pre_gamma=w[3], stats=stats, T=T, d=d, res_scale=0.5, branch_scale=2.0, dx=(a := new(T, d)),
                                                 dy=(b := new(T, d, dtype=bf)), d_post_gamma=(c := new(d)), d_post_beta=(e := new(d)),
                                                 d_gate=(f := new(d)), d_pre_gamma=(p := new(d)), d_pre_beta=(q := new(d)),
                                                 ws=room(_lib.OP_RESIDUAL_NORM_BWD, T, 1, 1, d)), (a, b, c, e, f, p, q))
    grad, start = n(1000), n(1000)

    def norm():
        keep = [start.clone(), grad, torch.zeros(1000, device="cuda"), torch.zeros(1000, device="cuda")]
        return dict(tensors=_table(keep), max_norm=1.0, norm=(o := new(2)), ws=room(_lib.OP_GRAD_NORM, 0, 1, 1)), (o, *keep)

    def step():
        keep = [start.clone(), grad, torch.zeros(1000, device="cuda"), torch.zeros(1000, device="cuda")]
        s = torch.zeros(2, dtype=torch.int32, device="cuda")
        return dict(tensors=_table(keep), state_bits=32, lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, seed=3, steps=s,
                    lr_scale=torch.full((1,), 0.5, device="cuda"), grad_scale=torch.full((1,), 0.25, device="cuda")), (*keep, s)

    yield "moe_grad_norm", norm
    yield "moe_adamw_step", step
    ids, weights = torch.randint(-1, E, (T, k), generator=g, device="cuda", dtype=torch.int32), n(T, k)
    packed = {}
    for name, m, N, K in (("ug", 2 * E, h, d), ("down", E, d, h)):
        packed[name] = room(_lib.OP_W4_WEIGHTS, 0, 1, m, K, N, group)
        groups = (K + group - 1) // group
        codes = torch.randint(0, 256, (m, N, (K + 1) // 2), generator=g, device="cuda", dtype=torch.uint8)
        _lib.moe_w4_pack(codes, n(m, N, groups, dtype=bf), None, m, N, K, group, packed[name])
    xb = n(T, d, dtype=bf)
    yield "moe_w4_matvec", lambda: (dict(x=xb, ids=ids, T=T, top_k=k, matrices=2 * E, N=h, K=d, group=group, packed=packed["ug"],
                                         y=(o := new(T * k, h))), (o,))
    yield "moe_w4_swiglu_decode", lambda: (dict(x=xb, ids=ids, weights=weights, T=T, top_k=k, E=E, d=d, h=h, group=group, w_ug=packed["ug"],
                                                w_down=packed["down"], out=(o := new(T, d, dtype=bf)), ws=room(_lib.OP_W4_DECODE, T, k, E, d, h)), (o,))


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
                fn(*[args[p] for p in order if p in args and p != "stream"])
            else:
                fn(**args, stream=torch.cuda.current_stream())
            results.append([o.clone() for o in outs])
        for other in results[1:]:
            assert all(torch.equal(a, b) for a, b in zip(results[0], other)), name
        # one argument wrong at a time: the same kind of error from both
        args, _ = make()
        for p, v in args.items():
            wrong = [v.cpu()] if isinstance(v, torch.Tensor) else [] if p in ("tensors", "seed") else [-5, "x"]
            if isinstance(v, torch.Tensor) and v.dim() == 2:
                wrong.append(v.t())
            for bad in wrong:
                if p in ("res_scale", "branch_scale", "lr") and bad == -5:
                    continue  # a number like any other
                kinds = []
                for fn in (python, compiled):
                    try:
                        fn(**{**make()[0], p: bad})
                        kinds.append(None)
                    except Exception as e:  # noqa: BLE001
                        kinds.append(type(e).__name__)
                kind = {"ArgumentError", "TypeError", "ValueError"}
                assert None not in kinds, (name, p, kinds)
                assert kinds[0] == kinds[1] or (isinstance(bad, str) and set(kinds) <= kind), (name, p, kinds)
        for fn in (python, compiled):
            with pytest.raises(TypeError):
                fn(**{**args, "nonsense": 1})
            with pytest.raises(TypeError):
                fn()
    assert seen == set(_lib.COMPILED_STEP)


def test_pointers_of_a_step(both):
    """Both loops write the same table, count the same versions and refuse the same."""
    p, c = [torch.zeros(5, device="cuda"), torch.zeros(9, dtype=torch.bfloat16, device="cuda")], [torch.zeros(5, dtype=torch.bfloat16, device="cuda"), None]
    g = [torch.zeros(5, dtype=torch.bfloat16, device="cuda"), torch.zeros(9, device="cuda")]
    tables = []
    for fn in (optim._pointers, _lib.adamw_pointers):
        opt = optim.AdamW(p, copies=c)
        before = [t._version for t in (*p, c[0])]
        fn(opt._table, 0, opt.params, opt.copies, g)
        assert [t._version for t in (*p, c[0])] == [v + 1 for v in before]
        tables.append([[getattr(q, f) for f in ("p", "copy", "g", "n", "p_dtype", "g_dtype")] for q in opt._table])
        for bad in ([g[0], g[1][:4]], [g[0].cpu(), g[1]], [g[0], g[1].double()], [g[0], g[1].half()]):
            with pytest.raises(ValueError):
                fn(opt._table, 0, opt.params, opt.copies, bad)
        with pytest.raises(ValueError):
            fn(opt._table, 0, [p[0], p[1].float()], opt.copies, g)
    assert tables[0] == tables[1]
