"""The residual join forward and backward against the fp64 reference.

Tolerances. As for the layer norm: a value is a handful of fp32 roundings (unit 2^-24) of terms no larger than its
scale, plus the errors of the row's mean and variance, 64 units of the terms' scale in all, rounded once. The
gradients pass the error of D on: dy takes it as the norm's backward takes its input. A weight gradient is a sum of T
terms added at most T / 608 + 64 deep, plus the terms' own errors."""
import numpy as np
import pytest
import torch

from oracle import train_oracle as R
from ragged_grouped_gemm_device_gb300 import _lib
from rounding import within_one_rounding

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
KINDS = {"none": 0, "layer": 1, "rms": 2}
EPS = 1e-5
GRADS = ("d_post_gamma", "d_post_beta", "d_gate", "d_pre_gamma", "d_pre_beta")


def _host(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _nan(*s, dtype=torch.float32):
    return torch.full(s, float("nan"), dtype=dtype, device="cuda")


class Case:
    def __init__(self, T, d, stream="bf16", branch="bf16", post="layer", pre="rms", w="fp32", gate=True, bias=True, branch_given=True,
                 offset=0.3, al=0.9, be=0.7, seed=0):
        g = torch.Generator().manual_seed(1000 * T + d + seed)
        n = lambda *s: torch.randn(*s, generator=g)
        self.T, self.d, self.post, self.pre, self.al, self.be = T, d, post, pre, al, be
        self.tx, self.ty = TYPES[stream], TYPES[branch]
        self.x, self.dr = ((n(T, d) + offset).to(self.tx).cuda() for _ in range(2))
        self.y = (0.6 * n(T, d) + offset).to(self.ty).cuda() if branch_given else None
        self.dn = n(T, d).to(self.ty).cuda() if pre != "none" else None
        wt = lambda on, mean: (mean + 0.3 * n(d)).to(TYPES[w]).cuda() if on else None
        self.pg, self.pb = wt(post != "none" and w != "none", 1.0), wt(post == "layer" and bias, 0.0)
        self.gate = wt(gate and branch_given, 0.5)
        self.qg, self.qb = wt(pre != "none", 1.0), wt(pre == "layer" and bias, 0.0)

    def forward(self, r=True, n=None, stats=True, x=None, y=None):
        x, y = self.x if x is None else x, self.y if y is None else y
        r = _nan(self.T, self.d, dtype=self.tx) if r is True else r
        if self.pre != "none" and n is None:
            n = _nan(self.T, self.d, dtype=self.ty)
        s = _nan(4, self.T) if stats else None
        _lib.moe_residual_norm_fwd(x, y, KINDS[self.post], self.pg, self.pb, self.gate, KINDS[self.pre], self.qg, self.qb, self.T,
                                   self.d, EPS, self.al, self.be, r, n, s)
        return r, n, s

    def backward(self, r, stats, dx=None, dy=None, dn=None, dr=None, y=None, grads=GRADS):
        dx = _nan(self.T, self.d, dtype=self.tx) if dx is None else dx
        y = self.y if y is None else y
        if y is not None and dy is None:
            dy = _nan(self.T, self.d, dtype=self.ty)
        allowed = [n for n in GRADS if (n in grads) and (self.pre != "none" or "pre" not in n)
                   and (self.post != "none" or "post" not in n) and (y is not None or n != "d_gate")]
        out = {n: _nan(self.d) for n in allowed}
        ws = _nan(max(1, _lib.moe_workspace_bytes(_lib.OP_RESIDUAL_NORM_BWD, self.T, 1, 1, self.d) // 4))
        _lib.moe_residual_norm_bwd(self.dn if dn is None else dn, self.dr if dr is None else dr, r if self.pre != "none" else None, y,
                                   KINDS[self.post], self.pg, self.pb, self.gate, KINDS[self.pre], self.qg, stats, self.T,
                                   self.d, self.al, self.be, dx, dy, **out, ws=ws)
        return {"dx": dx, "dy": dy, **out}

    def check_forward(self, r, n, stats):
        w = lambda t, fill: fill if t is None else np.abs(_host(t))
        x, y = _host(self.x), _host(self.y)
        ref, yhat, mean1, rstd1 = R.join(x, y, self.post, _host(self.pg), _host(self.pb), _host(self.gate), self.al, self.be, EPS)
        st = _host(stats)
        scale = abs(self.al) * np.abs(x)
        if y is not None:
            big = np.abs(y).max(axis=1)
            loss = 1 + (big * rstd1 if self.post != "none" else 0 * big)
            scale = scale + abs(self.be) * w(self.gate, 1.0) * ((np.abs(yhat) + 1) * w(self.pg, 1.0) * loss[:, None] + w(self.pb, 0.0))
            assert (np.abs(st[0] - mean1) <= 64 * U * big).all()
            assert (np.abs(st[1] - rstd1) <= 64 * U * rstd1 * loss).all()
        assert within_one_rounding(_host(r), ref, 64 * U * scale, self.tx)
        if self.pre == "none":
            return
        rh = _host(r)
        hat, mean2, rstd2 = R.norm(self.pre, rh, EPS)
        big = np.abs(rh).max(axis=1)
        loss = 1 + big * rstd2
        assert (np.abs(st[2] - mean2) <= 64 * U * big).all()
        assert (np.abs(st[3] - rstd2) <= 64 * U * rstd2 * loss).all()
        ref = hat * (1.0 if self.qg is None else _host(self.qg)) + (0.0 if self.qb is None else _host(self.qb))
        scale = (np.abs(hat) + 1) * w(self.qg, 1.0) * loss[:, None] + w(self.qb, 0.0)
        assert within_one_rounding(_host(n), ref, 64 * U * scale, self.ty)

    def check_backward(self, r, got, dn=None, dr=None):
        dn, dr = self.dn if dn is None else dn, self.dr if dr is None else dr
        w = lambda t, fill: fill if t is None else np.abs(_host(t))
        o = R.join_grad(_host(dn), _host(dr), _host(r), _host(self.y), self.post, _host(self.pg), _host(self.pb), _host(self.gate),
                        self.pre, _host(self.qg), self.al, self.be, EPS)

        def through(e, g, hat, rstd, rows, kind):
            """The error of a norm's backward whose input g has the error e."""
            if kind == "none":
                return e
            loss = (1 + np.abs(rows).max(axis=1) * rstd)[:, None]
            a = lambda v: v + v.mean(axis=1, keepdims=True) + (np.abs(hat) + 1) * (v * (np.abs(hat) + 1)).mean(axis=1, keepdims=True)
            return rstd[:, None] * (a(e) + 64 * U * a(np.abs(g)) * loss)

        eD = 64 * U * np.abs(o["D"])
        if dr is not None:
            eD = eD + 64 * U * np.abs(_host(dr))
        depth = self.T / 608 + 64
        if self.pre != "none":
            eD = eD + through(64 * U * np.abs(o["g2"]), o["g2"], o["rhat"], o["rstd2"], _host(r), self.pre)
            loss = (1 + np.abs(_host(r)).max(axis=1) * o["rstd2"])[:, None]
            dnh = np.abs(_host(dn))
            if "d_pre_gamma" in got:
                assert (np.abs(_host(got["d_pre_gamma"]) - o["d_pre_gamma"]) <= depth * U * (dnh * (np.abs(o["rhat"]) + 1) * loss).sum(axis=0)).all()
            if "d_pre_beta" in got:
                assert (np.abs(_host(got["d_pre_beta"]) - o["d_pre_beta"]) <= depth * U * dnh.sum(axis=0)).all()
        assert within_one_rounding(_host(got["dx"]), o["dx"], abs(self.al) * eD, self.tx)
        if self.y is None:
            return
        k = abs(self.be) * w(self.gate, 1.0)
        e1 = k * w(self.pg, 1.0) * (eD + 4 * U * np.abs(o["D"]))
        assert within_one_rounding(_host(got["dy"]), o["dy"], through(e1, o["g1"], o["yhat"], o["rstd1"], _host(self.y), self.post)
                                   + 4 * U * np.abs(o["dy"]), self.ty)
        loss = 1 + (np.abs(_host(self.y)).max(axis=1) * o["rstd1"])[:, None] * (self.post != "none")
        s1 = (eD * (np.abs(o["yhat"]) + 1) + depth * U * np.abs(o["D"]) * (np.abs(o["yhat"]) + 1) * loss).sum(axis=0)
        s0 = (eD + depth * U * np.abs(o["D"])).sum(axis=0)
        bounds = {"d_post_gamma": k * s1, "d_post_beta": k * s0, "d_gate": abs(self.be) * (w(self.pg, 1.0) * s1 + w(self.pb, 0.0) * s0)}
        for name, tol in bounds.items():
            if name in got:
                assert (np.abs(_host(got[name]) - o[name]) <= tol + 4 * U * np.abs(o[name])).all(), name

    def check(self):
        r, n, s = self.forward()
        self.check_forward(r, n, s)
        self.check_backward(r, self.backward(r, s))


NORMS = [("layer", "layer"), ("rms", "rms"), ("layer", "rms"), ("rms", "layer"), ("none", "layer"), ("none", "rms"), ("layer", "none"),
         ("rms", "none"), ("none", "none")]


# widths on both sides of each register layout's limit, odd ones, rows without registers; from one row to more
# than the backward's blocks
@pytest.mark.parametrize("stream,branch", [("bf16", "bf16"), ("fp32", "bf16"), ("fp32", "fp32")])
@pytest.mark.parametrize("T,d", [(1, 1), (1, 2048), (3, 8), (5, 31), (2, 127), (7, 256), (4, 264), (9, 512), (6, 1000), (3, 1001),
                                 (2, 2056), (3, 4096), (2, 4104), (2, 8191), (2, 8192), (1, 8200), (1, 16384), (2, 16392),
                                 (1, 40001), (700, 96), (1300, 2048), (2500, 65)])
def test_matches_the_reference(lib, T, d, stream, branch):
    Case(T, d, stream, branch, *NORMS[(T + d) % 4]).check()


@pytest.mark.parametrize("post,pre", NORMS)
@pytest.mark.parametrize("d", [65, 512, 2048, 20000])
def test_every_pair_of_norms(lib, d, post, pre):
    Case(37, d, "bf16", "bf16", post, pre, gate=(d != 512)).check()
    Case(5, d, "fp32", "bf16", post, pre, bias=False).check()


# rows off the 16-byte grid in every register layout, with several rows a block
@pytest.mark.parametrize("stream,branch", [("bf16", "bf16"), ("fp32", "bf16"), ("fp32", "fp32")])
@pytest.mark.parametrize("T,d", [(2100, 255), (2000, 257), (1900, 511), (1000, 513), (1000, 1023), (1000, 1025), (950, 2047), (400, 2049), (350, 4095),
                                 (310, 4097), (310, 7001)])
def test_odd_widths_of_every_layout(lib, T, d, stream, branch):
    Case(T, d, stream, branch, *NORMS[(T + d) % 4]).check()


# more than 32 rows a block: the backward fetches their statistics 32 rows at a time
@pytest.mark.parametrize("T,d", [(60000, 16), (60000, 9), (15000, 520), (15000, 521)])
def test_many_rows_a_block(lib, T, d):
    Case(T, d, "bf16", "bf16", "layer", "layer").check()


@pytest.mark.parametrize("w", ["bf16", "fp32"])
@pytest.mark.parametrize("d", [100, 1024])
def test_weights_of_both_types(lib, d, w):
    Case(33, d, "fp32", "bf16", "layer", "layer", w=w).check()


@pytest.mark.parametrize("d", [77, 1024, 16392])
def test_without_a_branch(lib, d):
    """The first norm of a model: n = pre(x), no rows of the branch; r need not be stored."""
    c = Case(9, d, "bf16", "bf16", "none", "rms", branch_given=False, al=1.0)
    r, n, s = c.forward()
    c.check_forward(r, n, s)
    assert torch.equal(r, c.x)
    _, n2, _ = c.forward(r=None)
    assert torch.equal(n, n2)
    got = c.backward(c.x, s)
    c.check_backward(c.x, got)
    assert got["dy"] is None


def test_r_is_not_stored(lib):
    for stream in ("bf16", "fp32"):
        for d in (130, 2048, 17000):
            c = Case(11, d, stream, "bf16", "rms", "layer")
            _, n, s = c.forward()
            _, n2, s2 = c.forward(r=None)
            assert torch.equal(n, n2) and torch.equal(s, s2)


@pytest.mark.parametrize("d", [520, 17008])
@pytest.mark.parametrize("stream,branch", [("bf16", "bf16"), ("fp32", "bf16"), ("fp32", "fp32")])
def test_rows_of_wider_buffers(lib, stream, branch, d):
    """Row pitches and bases that are no multiple of 16 bytes, and one upstream row for all tokens; then aligned rows of
    wider buffers. Nothing is written outside the rows."""
    T = 19
    c = Case(T, d, stream, branch, "layer", "rms")
    r0, n0, s0 = c.forward()
    g0 = c.backward(r0, s0)
    for pad, at in ((11, 3), (16, 8)):
        wide = lambda t: torch.cat([t.new_full((T, at), 9.0), t, t.new_full((T, pad - at), 9.0)], dim=1)
        view = lambda t: wide(t)[:, at:at + d]
        out = {n: torch.full((T, d + pad), float("nan"), dtype=t, device="cuda")
               for n, t in (("r", c.tx), ("n", c.ty), ("dx", c.tx), ("dy", c.ty))}
        cut = lambda n: out[n][:, at:at + d]
        r, n, s = c.forward(r=cut("r"), n=cut("n"), x=view(c.x), y=view(c.y))
        c.check_forward(r, n, s)
        got = c.backward(r, s, dx=cut("dx"), dy=cut("dy"), dn=view(c.dn), dr=view(c.dr), y=view(c.y))
        c.check_backward(r, got)
        for t in out.values():
            assert torch.isnan(t[:, :at]).all() and torch.isnan(t[:, at + d:]).all()
    one_n, one_r = c.dn[:1].expand(T, d), c.dr[:1].expand(T, d)
    got = c.backward(r0, s0, dn=one_n, dr=one_r)
    c.check_backward(r0, got, dn=one_n, dr=one_r)
    same = c.backward(r0, s0, dn=one_n.contiguous(), dr=one_r.contiguous())
    assert all(torch.equal(got[n], same[n]) for n in got)
    assert set(g0) == set(got)


@pytest.mark.parametrize("T,d", [(9, 1024), (5, 1001), (700, 256), (3, 17000)])
@pytest.mark.parametrize("stream,branch", [("bf16", "bf16"), ("fp32", "bf16")])
def test_outputs_over_inputs(lib, T, d, stream, branch):
    c = Case(T, d, stream, branch, "layer", "layer")
    r, n, s = c.forward()
    x, y = c.x.clone(), c.y.clone()
    r2, n2, s2 = c.forward(r=x, n=y, x=x, y=y)
    assert torch.equal(r, x) and torch.equal(n, y) and torch.equal(s, s2)
    want = c.backward(r, s)
    dr, dn = c.dr.clone(), c.dn.clone()
    got = c.backward(r, s, dx=dr, dy=dn, dr=dr, dn=dn)
    assert all(torch.equal(want[k], got[k]) for k in want)
    y = c.y.clone()
    got = c.backward(r, s, dy=y, y=y)
    assert all(torch.equal(want[k], got[k]) for k in want)
    r3 = r.clone()
    got = c.backward(r3, s, dx=r3)
    assert all(torch.equal(want[k], got[k]) for k in want)


def test_gradients_left_out(lib):
    c = Case(50, 300, "bf16", "bf16", "layer", "layer")
    r, _, s = c.forward()
    want = c.backward(r, s)
    for names in ((), ("d_gate",), ("d_post_gamma", "d_pre_beta")):
        got = c.backward(r, s, grads=names)
        assert set(names) <= set(got) and all(torch.equal(got[n], want[n]) for n in got)
    # no gradient from the residual path, and no dx wanted
    z = torch.zeros_like(c.dr)
    full = c.backward(r, s, dr=z)
    dy, dx, ws = torch.empty_like(c.y), torch.empty_like(c.x), _nan(_lib.moe_workspace_bytes(_lib.OP_RESIDUAL_NORM_BWD, 50, 1, 1, 300) // 4)
    _lib.moe_residual_norm_bwd(c.dn, None, r, c.y, 1, c.pg, c.pb, c.gate, 1, c.qg, s, 50, 300, c.al, c.be, None, dy, ws=ws)
    assert torch.equal(dy, full["dy"])
    _lib.moe_residual_norm_bwd(c.dn, None, r, c.y, 1, c.pg, c.pb, c.gate, 1, c.qg, s, 50, 300, c.al, c.be, dx, dy, ws=ws)
    assert torch.equal(dx, full["dx"])


def test_large_offsets_and_constant_rows(lib):
    Case(8, 768, "fp32", "fp32", "layer", "layer", offset=200.0).check()
    c = Case(4, 512, "fp32", "fp32", "layer", "layer", al=1.0, be=0.5)
    c.y[:] = 3.0           # variance 0: z = post_beta
    r, _, _ = c.forward()
    want = c.x + 0.5 * (c.gate * c.pb)
    assert (r - want).abs().max() <= 4 * U * (c.x.abs() + want.abs()).max()


def test_nan_and_infinity_stay_in_their_rows(lib):
    for d in (320, 17001):
        c = Case(6, d)
        r0, n0, s0 = c.forward()
        g0 = c.backward(r0, s0)
        c.y[2, 7], c.x[4, 0] = float("nan"), float("inf")
        r, n, s = c.forward()
        assert torch.isnan(r[2]).all() and torch.isnan(n[2]).all() and torch.isinf(r[4, 0])
        rest = [0, 1, 3, 5]
        assert torch.equal(r[rest], r0[rest]) and torch.equal(n[rest], n0[rest])
        g = c.backward(r, s)
        assert torch.equal(g["dx"][rest], g0["dx"][rest]) and torch.equal(g["dy"][rest], g0["dy"][rest])
        assert torch.isnan(g["dy"][2]).all()


def test_no_rows_and_repeated_calls(lib):
    c = Case(1, 64, post="layer", pre="layer")
    e = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    _lib.moe_residual_norm_fwd(e, e, 1, c.pg, c.pb, None, 1, c.qg, c.qb, 0, 64, EPS, 1.0, 1.0, e, e)
    out = [_nan(64) for _ in range(5)]
    _lib.moe_residual_norm_bwd(e, e, e, e, 1, c.pg, c.pb, c.gate, 1, c.qg, torch.empty(0, device="cuda"), 0, 64, 1.0, 1.0, e, e, *out)
    assert all((t == 0).all() for t in out)
    c = Case(5000, 512, post="rms", pre="layer")
    r, _, s = c.forward()
    a, b = c.backward(r, s), c.backward(r, s)
    assert all(torch.equal(a[k], b[k]) for k in a)


def test_on_another_stream_and_in_a_graph(lib):
    c = Case(64, 256)
    r0, n0, s0 = c.forward()
    want = c.backward(r0, s0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        r, n, s = c.forward()
        got = c.backward(r, s)
    side.synchronize()
    assert torch.equal(r, r0) and torch.equal(n, n0) and all(torch.equal(got[k], want[k]) for k in want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r, n, s = c.forward()
        got = c.backward(r, s)
    c.x.mul_(0.5)
    graph.replay()
    r1, n1, s1 = c.forward()
    want = c.backward(r1, s1)
    assert torch.equal(r, r1) and torch.equal(n, n1) and all(torch.equal(got[k], want[k]) for k in want)


def test_refusals(lib):
    c = Case(4, 64, post="layer", pre="layer")
    call = lambda **k: _lib.moe_residual_norm_fwd(**{**dict(
        x=c.x, y=c.y, post=1, post_gamma=c.pg, post_beta=c.pb, gate=c.gate, pre=1, pre_gamma=c.qg, pre_beta=c.qb, T=4, d=64, eps=EPS,
        res_scale=1.0, branch_scale=1.0, r=torch.empty_like(c.x), n=torch.empty_like(c.y)), **k})
    call()
    for bad in (dict(x=c.x.half()), dict(x=c.x.t()), dict(r=torch.empty(4, 64, device="cuda")), dict(n=torch.empty(4, 64, device="cuda")),
                dict(pre_gamma=c.qg.bfloat16()), dict(gate=c.gate[:32]), dict(x=c.x.cpu()), dict(T=5)):
        with pytest.raises(ValueError):
            call(**bad)
    for bad in (dict(post=3), dict(post=2), dict(pre=0), dict(n=None), dict(y=None), dict(eps=-1.0), dict(res_scale=float("nan")),
                dict(branch_scale=float("inf"))):
        with pytest.raises(_lib.MoEError):
            call(**bad)
