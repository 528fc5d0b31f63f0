"""Pins of the oracle's rotary table, norm + rotation and 8-bit integer linear layer against what their
definitions fix."""
from fractions import Fraction

import numpy as np

import oracle


def test_rope_angles_by_hand_and_axis_order():
    pos = np.array([[3.0, -2.0], [0.0, 0.5]])
    a = oracle.rope_angles(pos, (4, 2), (100.0, 10000.0))
    # axis 0: frequencies 1 and 100^-0.5 = 0.1; axis 1: frequency 1
    assert np.allclose(a, [[3.0, 0.3, -2.0], [0.0, 0.0, 0.5]], rtol=1e-15, atol=0)


def test_norm_rope_keeps_lengths_and_relative_angles():
    """Unit weights: the norm gives rows of length sqrt(D); a rotation keeps it, and the dot product of
    two rotated rows depends on the difference of their positions only."""
    rng = np.random.default_rng(1)
    D = 16
    q, k = rng.normal(size=(1, 1, 1, D)), rng.normal(size=(1, 1, 1, D))
    w = np.ones(D)

    def at(x, p, inter):
        a = oracle.rope_angles(np.array([[float(p)]]), (D,), (50.0,))
        return oracle.norm_rope(x, w, np.stack([np.cos(a), np.sin(a)], -1), 0.0, inter)[0].reshape(-1)

    for inter in (True, False):
        assert abs(np.linalg.norm(at(q, 5, inter)) - np.sqrt(D)) < 1e-12
        assert abs(at(q, 5, inter) @ at(k, 2, inter) - at(q, 13, inter) @ at(k, 10, inter)) < 1e-12
        assert abs(at(q, 5, inter) @ at(k, 2, inter) - at(q, 5, inter) @ at(k, 3, inter)) > 1e-3


def test_norm_rope_quarter_turn_pairs_partial_and_layout():
    x = np.arange(1.0, 2 * 3 * 8 + 1).reshape(1, 2, 3, 8)
    table = np.zeros((2, 2, 2))
    table[..., 1] = 1.0                              # cos 0, sin 1: (a, b) -> (-b, a)
    y, _ = oracle.norm_rope(x, None, table, 1e-6, True)
    assert y.shape == (1, 3, 2, 8)
    assert np.array_equal(y[0, 1, 1], [-34.0, 33.0, -36.0, 35.0, 37.0, 38.0, 39.0, 40.0])
    y, _ = oracle.norm_rope(x, None, table, 1e-6, False)
    assert np.array_equal(y[0, 1, 1], [-35.0, -36.0, 33.0, 34.0, 37.0, 38.0, 39.0, 40.0])


def test_quantize_int8_rows_against_fractions():
    rng = np.random.default_rng(2)
    x = (rng.normal(size=(4, 64)) * 2.0 ** rng.integers(-6, 6, size=(4, 64))).astype(np.float16)
    x[1] = 0
    x[2, :4] = [8.0, -8.0, 4.0, -4.0]                # 127 * 4 / 8 = 63.5: a tie
    x[2, 4:] = 0
    codes, scale = oracle.quantize_int8_rows(x)
    assert scale[1] == 1.0 and not codes[1].any()
    assert list(codes[2, :4]) == [127, -127, 64, -64]
    for m in range(4):
        top = max(abs(Fraction(float(v))) for v in x[m])
        for k in range(64):
            if top:
                assert codes[m, k] == round(Fraction(float(x[m, k])) * 127 / top)   # Fraction: ties to even


def test_gemm_int8_triple_loop_and_extremes():
    rng = np.random.default_rng(3)
    a, b = rng.integers(-128, 128, size=(3, 5)), rng.integers(-128, 128, size=(4, 5))
    y, size = oracle.gemm_int8(a.astype(np.int8), b.astype(np.int8), np.full(3, 0.5), np.full(4, 0.25), np.arange(4.0))
    for m in range(3):
        for n in range(4):
            s = sum(int(a[m, k]) * int(b[n, k]) for k in range(5)) * 0.125
            assert y[m, n] == s + n and size[m, n] == abs(s) + n
    low = np.full((1, 131071), -128, np.int8)
    assert oracle.gemm_int8(low, low, [1.0], [1.0])[0][0, 0] == 131071 * 16384 < 2 ** 31
