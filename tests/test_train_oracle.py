"""The fp64 references of the residual join, AdamW's 8-bit states and the 4-bit integers, against differences,
hand-worked values and their definitions."""
import itertools

import numpy as np
import pytest

from oracle import train_oracle as R


@pytest.mark.parametrize("post,pre", list(itertools.product(["none", "layer", "rms"], repeat=2)))
def test_join_gradients_against_differences(post, pre):
    rng = np.random.default_rng(5)
    T, d, eps, al, be = 3, 6, 1e-2, 0.8, -1.3
    n = lambda *s: rng.standard_normal(s)
    x, y, dn, dr = n(T, d), n(T, d), n(T, d), n(T, d)
    w = dict(pg=1 + 0.3 * n(d), pb=n(d) if post == "layer" else None, gate=n(d), qg=1 + 0.3 * n(d), qb=n(d) if pre == "layer" else None)
    if post == "none":
        w["pg"] = None
    if pre == "none":
        w["qg"], dn = None, None

    def loss(x, y, w):
        r, *_ = R.join(x, y, post, w["pg"], w["pb"], w["gate"], al, be, eps)
        s = (r * dr).sum()
        if pre != "none":
            hat, _, _ = R.norm(pre, r, eps)
            s += ((hat * w["qg"] + (0 if w["qb"] is None else w["qb"])) * dn).sum()
        return s

    r, *_ = R.join(x, y, post, w["pg"], w["pb"], w["gate"], al, be, eps)
    o = R.join_grad(dn, dr, r, y, post, w["pg"], w["pb"], w["gate"], pre, w["qg"], al, be, eps)

    def diff(t, f):
        g = np.zeros_like(t)
        for i in np.ndindex(*t.shape):
            h = 1e-6
            a, b = t.copy(), t.copy()
            a[i] += h
            b[i] -= h
            g[i] = (f(a) - f(b)) / (2 * h)
        return g

    close = lambda a, b: np.testing.assert_allclose(a, b, rtol=1e-6, atol=1e-7)
    close(o["dx"], diff(x, lambda v: loss(v, y, w)))
    close(o["dy"], diff(y, lambda v: loss(x, v, w)))
    for key, name in (("pg", "d_post_gamma"), ("pb", "d_post_beta"), ("gate", "d_gate"), ("qg", "d_pre_gamma"), ("qb", "d_pre_beta")):
        if w[key] is not None:
            close(o[name], diff(w[key], lambda v: loss(x, y, {**w, key: v})))


def test_scales_and_elements_of_the_8_bit_states():
    x = np.zeros(96)
    x[0] = 448.0            # just fits 2^0
    x[33] = 449.0           # does not: 2^1
    s = R.scale_exponent(x)
    assert s.tolist() == [0, 1, -127]
    x[1], x[2], x[34] = 0.30, -17.0, 2.0 ** -20
    q, s, _ = R.quantize8(x, np.zeros(96), False)
    assert q[1] == 0.28125 and q[2] == -16.0 and q[34] == 0.0       # steps 1/32 and 2, and less than half the lowest step
    q, _, _ = R.quantize8(x, np.full(96, 0.999), True)
    assert q[1] == 0.3125 and q[2] == -18.0 and q[34] == 2.0 ** -9 and q[3] == 0.0
    # unbiased: the mean over u of what 0.30 becomes is 0.30
    u = np.arange(4096) / 4096
    assert abs(R.round_up_where(np.full(4096, 0.30), u, 3, -6)[0].mean() - 0.30) < 1 / 32 / 4096 + 1e-12


def test_mix_is_a_bijection_with_known_values():
    assert R.mix(0) == 0 and int(R.mix(1)) == 0x514E28B7
    v = R.mix(np.arange(1 << 16))
    assert np.unique(v).size == 1 << 16
    assert abs((v & np.uint64(0xFFFF)).mean() / 65535 - 0.5) < 0.01


def test_adamw_by_hand():
    p, m, v = R.adamw(np.array([1.0]), np.array([2.0]), np.zeros(1), np.zeros(1), 1, 0.1, 0.9, 0.99, 0.0, 0.5)
    assert np.allclose(m, 0.2) and np.allclose(v, 0.04) and np.allclose(p, 0.95 - 0.1)  # the first step has size lr


def test_four_bit_round_trip_and_packing():
    rng = np.random.default_rng(1)
    w = R.to_bf16(rng.standard_normal((5, 77)).astype(np.float32))
    w[3, 32:64] = 0.0
    for group in (32, 64, 128):
        c, s, z = R.quantize4(w, group)
        back = R.dequantize4(c, s, z, group)
        step = np.repeat(s, group, axis=1)[:, :77]
        # half a step, and one more for what the rounded scale and zero point clip at the ends
        assert (np.abs(back - w) <= 1.5 * step).all() and (c <= 15).all()
    assert (R.quantize4(w, 32)[1][3, 1] == 0) and (R.dequantize4(*R.quantize4(w, 32), 32)[3, 32:64] == 0).all()
    codes = rng.integers(0, 16, (2, 17, 130)).astype(np.uint8)
    packed = R.pack4(codes, np.ones((2, 17, 5), np.uint16), np.full((2, 17, 5), 3, np.uint8), 32)
    tiles, chunks = 2, 2
    # matrix 1, row 16 (tile 1, row 0), chunk 1, word 0 of quarter 0, which is rotated left by 3 bits
    at = ((1 * tiles + 1) * chunks + 1) * (1024 + 128 + 32)
    word = int(packed[at:at + 4].view(np.uint32)[0])
    word = word >> 3 | (word & 7) << 29
    assert word & 15 == codes[1, 16, 128] and (word >> 16) & 15 == codes[1, 16, 129]
    # past the row's end in its last group: the zero point
    assert (word >> 4) & 15 == 3
