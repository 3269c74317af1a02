"""The MX4 oracle against brute force in exact arithmetic (CPU)."""

from fractions import Fraction

import numpy as np
import pytest

from oracle import mx4_oracle as mx

GRID = [Fraction(0), Fraction(1, 2), Fraction(1), Fraction(3, 2), Fraction(2), Fraction(3), Fraction(4), Fraction(6)]


def brute_code(v: float, s: int) -> int:
    a = abs(Fraction(v)) / Fraction(2) ** s
    best = min(range(8), key=lambda i: (abs(GRID[i] - a), i % 2))
    return best + (8 if np.signbit(v) else 0)


def brute_scale(block) -> int:
    top = max(abs(Fraction(float(v))) for v in block)
    if top == 0:
        return -127
    s = -200
    while Fraction(2) ** (s + 1) <= top:
        s += 1
    return max(-127, min(127, s - 2))


@pytest.mark.parametrize("seed", range(4))
def test_quantize_against_fractions(seed):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((4, 48)) * 2.0 ** rng.integers(-30, 15, (4, 48))
    x = x.astype(np.float16).astype(np.float64)
    x[0, :5] = [0.0, -0.0, 65504.0, -65504.0, 2.0 ** -24]
    x[1, :32] = 0.0
    # every midpoint of the grid and its neighbours, under a block maximum of 4
    x[2, :16] = [4, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5, 7.75]
    codes, scales = mx.mx4_quantize(x)
    for r in range(4):
        for b in range(2):
            block = x[r, 32 * b:32 * b + 32]
            s = brute_scale(block)
            assert scales[r, b] == s + 127
            assert [int(c) for c in codes[r, 32 * b:32 * b + 32]] == [brute_code(v, s) for v in block]


def test_ties_and_saturation():
    x = np.zeros((1, 32))
    x[0, :9] = [4, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.96875]
    v = mx.mx4_round(x)
    assert v[0, :9].tolist() == [4, 0, 1, 1, 2, 2, 4, 4, 6]


def test_nonfinite_blocks_and_layout():
    x = np.ones((2, 80))
    x[0, 3], x[1, 70] = np.inf, np.nan
    codes, scales = mx.mx4_quantize(x)
    assert scales.tolist() == [[255, 125, 125], [125, 125, 255]]
    assert codes[0, :32].max() == 0 and codes[1, 64:].max() == 0
    v = mx.mx4_values(codes, scales)
    assert np.isnan(v[0, :32]).all() and np.isnan(v[1, 64:]).all()
    assert (v[0, 32:] == 1).all() and (v[1, :64] == 1).all()
    p = mx.mx4_pack(codes)
    assert p.shape == (2, 48) and p[0, 16] == (codes[0, 32] | codes[0, 33] << 4) and (p[:, 40:] == 0).all()


def test_scaling_by_powers_of_two_moves_the_scale_alone():
    rng = np.random.default_rng(5)
    x = rng.standard_normal((3, 64))
    c0, s0 = mx.mx4_quantize(x)
    c1, s1 = mx.mx4_quantize(x * 2.0 ** 9)
    assert (c0 == c1).all() and (s1 == s0 + 9).all()


def test_route_ties_masks_and_norms():
    inf = np.inf
    logits = np.array([[1.0, 3.0, 3.0, -inf, 2.0], [-inf] * 5, [-inf, 0.0, -inf, -inf, -inf], [0.0, np.nan, 1.0, 9.0, 2.0]])
    ids, w = mx.moe_route(logits, 3, True)
    assert ids.tolist() == [[1, 2, 4], [-1, -1, -1], [1, -1, -1], [1, 3, 4]]
    assert np.allclose(w[:3].sum(1), [1, 0, 1]) and np.isnan(w[3]).all()
    _, w = mx.moe_route(logits, 3, False)
    e = np.exp([1.0, 3.0, 3.0, 2.0])
    assert np.allclose(w[0], np.array([np.exp(3), np.exp(3), np.exp(2)]) / e.sum())


def test_moe_layer_of_one_expert_is_a_gated_product():
    rng = np.random.default_rng(2)
    X, gu, dn = rng.standard_normal((3, 32)), rng.standard_normal((1, 32, 32)), rng.standard_normal((1, 32, 16))
    y, ids, w, bound = mx.moe_layer(X, np.zeros((3, 1)), gu, dn, 1, True)
    g, u = (gu[0] @ X.T)[:16], (gu[0] @ X.T)[16:]
    assert np.allclose(y, (dn[0] @ (g / (1 + np.exp(-g)) * u)).T)
    assert (ids == 0).all() and (w == 1).all() and (bound > 0).all() and bound.max() < 1e-3 * np.abs(y).max()
