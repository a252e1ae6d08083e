"""Host-side refusals of the residual join, AdamW and 4-bit integer entry points, and their workspace sizes (no GPU: validation
fails before any CUDA call)."""
import ctypes

import pytest

from ragged_grouped_gemm_device_gb300 import _lib, build

INVALID, SHAPE, WS = 1, 2, 3
BIG = 1 << 30


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


p, p2, p3 = ctypes.c_void_p(256), ctypes.c_void_p(258), ctypes.c_void_p(257)  # never dereferenced


def test_workspaces():
    build.build()
    wb = _lib.moe_workspace_bytes
    # four fp32 partial rows for each of at most 608 blocks, two floats a row
    assert wb(_lib.OP_RESIDUAL_NORM_BWD, 16384, 1, 1, 2048) == 608 * 4 * 2048 * 4 + 16384 * 8
    assert wb(_lib.OP_RESIDUAL_NORM_BWD, 5, 1, 1, 100) == 5 * 4 * 100 * 4 + 5 * 8
    assert wb(_lib.OP_RESIDUAL_NORM_BWD, 5, 1, 1, 0) == 0 and wb(_lib.OP_RESIDUAL_NORM_BWD, 5, 1, 1, (1 << 20) + 1) == 0
    assert wb(_lib.OP_GRAD_NORM, 0, 1, 1) > 0
    # pieces of 16 rows by 128 elements: 1024 bytes of codes, then the groups' scales and zero points, in multiples of 16 bytes
    n = 256 * 48 * 16
    assert wb(_lib.OP_W4_WEIGHTS, 0, 1, 256, 2048, 768, 128) == n * (1024 + 32 + 16)
    assert wb(_lib.OP_W4_WEIGHTS, 0, 1, 2048, 33, 17, 32) == 2048 * 2 * (1024 + 128 + 32)
    assert wb(_lib.OP_W4_WEIGHTS, 0, 1, 1, 1, 1, 32) == (1024 + 128 + 32 + 255) // 256 * 256
    for bad in ((0, 64, 64, 32), (2049, 64, 64, 32), (4, 0, 64, 32), (4, 64, 0, 32), (4, 64, 64, 48), (4, 64, 64, 0), (4, (1 << 20) + 1, 64, 32)):
        E, d, h, group = bad
        assert wb(_lib.OP_W4_WEIGHTS, 0, 1, E, d, h, group) == 0
    assert wb(_lib.OP_W4_DECODE, 16, 8, 128, 2048, 768) > 0 and wb(_lib.OP_W4_DECODE, 4097, 1, 128, 2048, 768) == 0


def test_residual_norm_refusals(lib):
    names = "x x_dtype ldx y y_dtype ldy post pg pb gate pre qg qb w T d eps al be r ldr n ldn stats stream".split()
    good = dict(x=p, x_dtype=0, ldx=64, y=p, y_dtype=0, ldy=64, post=1, pg=p, pb=p, gate=p, pre=2, qg=p, qb=None, w=1, T=4, d=64, eps=1e-5,
                al=1.0, be=1.0, r=p, ldr=64, n=p, ldn=64, stats=p, stream=None)
    f = lambda **k: lib.moe_residual_norm_fwd(*[{**good, **k}[n] for n in names])
    for bad in (dict(T=-1), dict(d=0), dict(x_dtype=2), dict(x_dtype=0, y_dtype=1), dict(w=3), dict(post=3), dict(pre=-1), dict(ldx=-1),
                dict(ldy=-1), dict(ldr=63), dict(ldn=63), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(al=float("nan")),
                dict(be=float("inf")), dict(x=None), dict(n=None), dict(pre=0), dict(y=None), dict(post=0), dict(post=2), dict(qb=p),
                dict(post=0, pg=None), dict(x=p3), dict(n=p3), dict(x_dtype=1, r=p2), dict(pg=p2), dict(stats=p2), dict(r=None, n=None, pre=0, qg=None)):
        assert f(**bad) == INVALID, bad
    assert f(d=(1 << 20) + 1, ldr=1 << 21, ldn=1 << 21) == SHAPE

    names = ("dn lddn dr lddr r ldr x_dtype y ldy y_dtype post pg pb gate pre qg w stats T d al be dx lddx dy lddy_out g0 g1 g2 g3 g4 ws "
             "n stream").split()
    good = dict(dn=p, lddn=64, dr=p, lddr=64, r=p, ldr=64, x_dtype=0, y=p, ldy=64, y_dtype=0, post=1, pg=p, pb=p, gate=p, pre=2, qg=p, w=1,
                stats=p, T=4, d=64, al=1.0, be=1.0, dx=p, lddx=64, dy=p, lddy_out=64, g0=p, g1=p, g2=p, g3=p, g4=p, ws=p, n=BIG, stream=None)
    f = lambda **k: lib.moe_residual_norm_bwd(*[{**good, **k}[n] for n in names])
    for bad in (dict(T=-1), dict(d=0), dict(x_dtype=0, y_dtype=1), dict(post=4), dict(pre=0), dict(dn=None), dict(r=None), dict(stats=None),
                dict(y=None), dict(dy=None), dict(lddx=63), dict(lddy_out=63), dict(lddr=-1), dict(post=0), dict(post=2), dict(dx=p3), dict(g2=p2),
                dict(ws=p2), dict(ws=None), dict(al=float("nan")), dict(dr=None, dn=None, pre=0, qg=None, g3=None, g4=None),
                dict(y=None, dy=None, post=0, pg=None, pb=None, gate=None, g0=None, g1=None)):
        assert f(**bad) == INVALID, bad
    assert f(n=_lib.moe_workspace_bytes(_lib.OP_RESIDUAL_NORM_BWD, 4, 1, 1, 64) - 1) == WS


def _tensor(**k):
    t = _lib.AdamWTensor(p=256, copy=None, g=256, m=256, v=256, m_scale=256, v_scale=256, n=100, weight_decay=0.1, p_dtype=1, g_dtype=1, reserved=0)
    for n, v in k.items():
        setattr(t, n, v)
    return (_lib.AdamWTensor * 1)(t)


def test_adamw_refusals(lib):
    assert ctypes.sizeof(_lib.AdamWTensor) == 80
    f = lambda t, count=1, bits=32, lr=1e-3, b1=0.9, b2=0.99, eps=1e-8, steps=p, ls=None, gs=None: lib.moe_adamw_step(
        t, count, bits, lr, b1, b2, eps, 0, steps, ls, gs, None)
    t = _tensor()
    for bad in (dict(bits=16), dict(lr=float("nan")), dict(b1=1.0), dict(b1=-0.1), dict(b2=1.0), dict(b2=float("nan")), dict(eps=-1e-8),
                dict(eps=float("inf")), dict(steps=None), dict(steps=p2), dict(ls=p2), dict(gs=p3), dict(count=-1)):
        assert f(t, **bad) == INVALID, bad
    assert f(None) == INVALID
    for bad in (dict(n=-1), dict(p=None), dict(g=None), dict(m=None), dict(v=None), dict(p_dtype=2), dict(g_dtype=-1), dict(reserved=1),
                dict(weight_decay=float("nan")), dict(p=258), dict(g=258), dict(m=258), dict(copy=257), dict(copy=256, p_dtype=0)):
        assert f(_tensor(**bad)) == INVALID, bad
    for bad in (dict(m_scale=None), dict(v_scale=None)):
        assert f(_tensor(**bad), bits=8) == INVALID
    assert f(_tensor(n=1 << 43)) == SHAPE

    g = lambda t, count=1, most=1.0, norm=p, ws=p, n=BIG: lib.moe_grad_norm(t, count, most, norm, ws, n, None)
    for bad in (dict(most=0.0), dict(most=-1.0), dict(most=float("nan")), dict(most=float("inf")), dict(norm=None), dict(norm=p2), dict(ws=None),
                dict(ws=p2), dict(count=-1)):
        assert g(t, **bad) == INVALID, bad
    assert g(t, n=8) == WS
    assert g(_tensor(g=258)) == INVALID and g(_tensor(n=1 << 43)) == SHAPE


def test_w4_refusals(lib):
    q = lambda w=p, rows=4, K=64, group=32, c=p, s=p, z=p: lib.moe_w4_quantize_rows(w, rows, K, group, c, s, z, None)
    for bad in (dict(rows=-1), dict(K=0), dict(w=None), dict(c=None), dict(s=None), dict(z=None), dict(w=p3), dict(s=p3)):
        assert q(**bad) == INVALID, bad
    assert q(group=16) == SHAPE and q(K=(1 << 20) + 1) == SHAPE and q(rows=1 << 31) == SHAPE
    k = lambda c=p, s=p, z=p, m=2, N=16, K=64, group=32, w=p, n=BIG: lib.moe_w4_pack(c, s, z, m, N, K, group, w, n, None)
    for bad in (dict(m=0), dict(N=0), dict(K=0), dict(c=None), dict(s=None), dict(w=None), dict(s=p3), dict(w=ctypes.c_void_p(128))):
        assert k(**bad) == INVALID, bad
    assert k(m=2049) == SHAPE and k(group=100) == SHAPE and k(n=_lib.moe_workspace_bytes(_lib.OP_W4_WEIGHTS, 0, 1, 2, 64, 16, 32) - 1) == WS
    v = lambda x=p, ldx=64, ids=p, T=2, top_k=2, m=3, N=16, K=64, group=32, w=p, y=p, t=0, ldy=16: lib.moe_w4_matvec(
        x, ldx, ids, T, top_k, m, N, K, group, w, y, t, ldy, None)
    for bad in (dict(T=-1), dict(top_k=0), dict(m=0), dict(ldx=-1), dict(ldy=15), dict(t=2), dict(x=None), dict(w=None), dict(y=None), dict(x=p3),
                dict(ids=p2), dict(t=1, y=p2), dict(w=ctypes.c_void_p(128))):
        assert v(**bad) == INVALID, bad
    assert v(top_k=33) == SHAPE and v(T=4097, top_k=1) == SHAPE and v(m=2049) == SHAPE and v(group=33) == SHAPE
    e = lambda x=p, ldx=64, ids=p, w=p, T=2, top_k=2, E=3, d=64, h=32, group=32, ug=p, dn=p, out=p, ldo=64, ws=p, n=BIG: lib.moe_w4_swiglu_decode(
        x, ldx, ids, w, T, top_k, E, d, h, group, ug, dn, out, ldo, ws, n, None)
    for bad in (dict(T=-1), dict(top_k=0), dict(E=0), dict(d=0), dict(h=0), dict(ldx=-1), dict(ldo=63), dict(x=None), dict(ids=None), dict(ug=None),
                dict(dn=None), dict(out=None), dict(ws=None), dict(x=p3), dict(w=p2), dict(out=p3), dict(ws=ctypes.c_void_p(64))):
        assert e(**bad) == INVALID, bad
    assert e(E=1025) == SHAPE and e(T=4097, top_k=1) == SHAPE and e(group=8) == SHAPE
    assert e(n=_lib.moe_workspace_bytes(_lib.OP_W4_DECODE, 2, 2, 3, 64, 32) - 1) == WS


def test_binding_without_an_entry_point(tmp_path):
    """An extension that is bound to a table without an entry point refuses its call instead of jumping nowhere."""
    import importlib.util
    import shutil

    path = build.build_binding()
    if path is None:
        pytest.skip("no compiler or headers for the extension")
    shutil.copy(path, tmp_path / "_binding.so")
    spec = importlib.util.spec_from_file_location("_binding", tmp_path / "_binding.so")
    binding = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(binding)
    binding.bind({n: 1 for n in _lib.COMPILED + ("moe_workspace_bytes",)}, _lib._check)
    with pytest.raises(RuntimeError, match="not bound"):
        binding.moe_w4_matvec(*[None] * 10)
    with pytest.raises(KeyError):
        binding.bind({n: 1 for n in _lib.COMPILED}, _lib._check)
