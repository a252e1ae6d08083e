"""Pins of the fp64 references of the layer norm, the gate and MXFP4: gradients against central
differences, the format against the values its definition gives."""
import numpy as np
import pytest

from oracle import block_oracle as B
from oracle import mx4_oracle as Q


def _difference(f, x, step=1e-6):
    out = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        a, b = x.copy(), x.copy()
        a[i] += step
        b[i] -= step
        out[i] = (f(a) - f(b)) / (2 * step)
    return out


@pytest.mark.parametrize("affine", [True, False])
def test_layer_norm_gradient_against_differences(affine):
    rng = np.random.default_rng(1)
    x, dy = rng.standard_normal((3, 7)), rng.standard_normal((3, 7))
    gamma, beta = (rng.standard_normal(7), rng.standard_normal(7)) if affine else (None, None)
    f = lambda x_, g_=gamma, b_=beta: (dy * B.layer_norm(x_, g_, b_, 1e-3)[0]).sum()
    dx, dg, db = B.layer_norm_grad(dy, x, gamma, 1e-3)
    # central differences of a smooth function: error of order step^2 and 1e-16 / step
    assert np.abs(dx - _difference(f, x)).max() < 1e-7
    if affine:
        assert np.abs(dg - _difference(lambda g: f(x, g), gamma)).max() < 1e-7
        assert np.abs(db - _difference(lambda b: f(x, gamma, b), beta)).max() < 1e-7


@pytest.mark.parametrize("renorm", [True, False])
def test_gate_gradient_against_differences(renorm):
    rng = np.random.default_rng(2)
    T, E, k = 5, 9, 3
    lg = rng.standard_normal((T, E))
    lg[1, 2:5] = -np.inf
    mask = np.array([1, 1, 0, 1, 1], bool)
    dw, dl = rng.standard_normal((T, k)), np.array([0.7, -0.3])

    def f(l_):
        g = B.gate(l_, mask, k, renorm)
        return (dw * g["weights"]).sum() + (dl * g["loss"]).sum()

    got, mag = B.gate_grad(B.gate(lg, mask, k, renorm), k, renorm, dw, dl)
    finite = np.isfinite(lg)
    want = np.zeros_like(lg)
    for i in zip(*np.nonzero(finite)):
        a, b = lg.copy(), lg.copy()
        a[i] += 1e-6
        b[i] -= 1e-6
        want[i] = (f(a) - f(b)) / 2e-6
    assert np.abs(got - want).max() < 1e-7
    assert (got[2] == 0).all() and (got[~finite] == 0).all()
    assert (np.abs(got) <= mag + 1e-15).all()


def test_gate_by_hand():
    lg = np.log(np.array([[1.0, 4.0, 2.0, 1.0], [2.0, 2.0, 2.0, 2.0]]))
    g = B.gate(lg, None, 2, False)
    assert g["ids"].tolist() == [[1, 2], [0, 1]]                    # ties to the lower expert
    assert np.allclose(g["weights"], [[0.5, 0.25], [0.25, 0.25]])
    assert np.allclose(B.gate(lg, None, 2, True)["weights"], [[2 / 3, 1 / 3], [0.5, 0.5]])
    assert g["counts"].tolist() == [1, 2, 1, 0] and g["n"] == 2
    # E sum f_e P_e = 4 (1/4 * (1/8 + 1/4) + 2/4 * (1/2 + 1/4) + 1/4 * (1/4 + 1/4)) / 2
    assert np.isclose(g["loss"][0], 4 * (0.25 * 0.375 + 0.5 * 0.75 + 0.25 * 0.5) / 2)
    assert np.isclose(g["loss"][1], np.log(8.0) ** 2)
    none = B.gate(np.full((2, 4), -np.inf), None, 2, True)
    assert (none["ids"] == -1).all() and none["n"] == 0 and (none["loss"] == 0).all()


def test_mxfp4_values_and_ties():
    v = np.zeros(32)
    v[:11] = [4.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.9, -0.3, -5.0]  # max 7.9: scale 2^0
    codes, scale = Q.quantize(v)
    assert scale.tolist() == [127]
    assert Q.values(codes, scale)[:11].tolist() == [4.0, 0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, 6.0, -0.5, -4.0]
    v[0] = np.nan
    assert Q.quantize(v)[1][0] == 255 and np.isnan(Q.fake_quant(v)).all()
    assert Q.quantize(np.zeros(32))[1][0] == 0
    # every code is its own quantization at every power of two
    for e in (-120, -3, 0, 17, 120):
        w = np.concatenate([Q.MAGNITUDES, -Q.MAGNITUDES, Q.MAGNITUDES, -Q.MAGNITUDES]) * 2.0 ** e
        assert (Q.fake_quant(w) == w).all()
