"""The reference of rules, MXFP4 and row statistics (oracle/shaped.py), pinned by values worked
out by hand."""
import math

import numpy as np

import oracle.shaped as S


def test_mx4_hand_worked_block():
    x = np.zeros((1, 32))
    # largest 7 -> exponent 2 -> e = 0: codes are those of the values themselves
    x[0, :12] = [7, 6, 5, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, 0.26, -5.01, -0.0]
    codes, scales = S.mx4_codes(x)
    assert scales[0, 0] == 127
    assert codes[0, :12].tolist() == [7, 7, 6, 6, 4, 4, 2, 2, 0, 1, 15, 8]
    assert S.mx4_values(codes, scales)[0, :12].tolist() == [6, 6, 4, 4, 2, 2, 1, 1, 0, 0.5, -6, 0]


def test_mx4_scales():
    x = np.zeros((4, 32))
    x[0, 3] = 1.0                      # floor(log2 1) - 2 = -2
    x[1, 0] = 2.0 ** -126              # clamped to -127
    x[2, 5] = np.inf
    codes, scales = S.mx4_codes(x)
    assert scales[:, 0].tolist() == [125, 0, 255, 0]
    assert codes[0, 3] == 6 and codes[1, 0] == 4 and np.isnan(S.mx4_values(codes, scales)[2]).all()


def test_rules_hand_worked():
    z = np.array([[2.0, -1.0, 0.5, 3.0]])
    out = S.shape_logits(z, np.array([0]), np.array([0]), 4, bias=np.array([0, 0, 1.0, 0]),
                         counts=np.array([[2, 1, 0, 0]]), repetition=np.array([2.0]),
                         presence=np.array([0.25]), frequency=np.array([0.5]),
                         allow=S.pack_bits(np.array([[1, 1, 1, 0]], dtype=bool)))
    # 2/2 - .25 - 1 = -.25;  -1*2 - .25 - .5 = -2.75;  .5 + 1;  banned
    assert out.tolist() == [[-0.25, -2.75, 1.5, -math.inf]]


def test_bits_round_trip():
    bits = np.random.default_rng(0).random((3, 77)) < 0.4
    assert (S.unpack_bits(S.pack_bits(bits), 77) == bits).all()
    assert S.pack_bits(np.ones((1, 32), dtype=bool)).tolist() == [[-1]]


def test_row_stats():
    z = np.array([[0.0, math.log(3.0), -np.inf], [-np.inf] * 3, [-np.inf, 5.0, -np.inf]])
    r = S.row_stats(z)
    assert r["tok"].tolist() == [1, -1, 1]
    np.testing.assert_allclose(r["conf"], [0.75, 0, 1])
    np.testing.assert_allclose(r["lse"], [math.log(4), -math.inf, 5.0])
    np.testing.assert_allclose(r["margin"], [0.5, 0, 1])
    np.testing.assert_allclose(r["entropy"], [0.75 * math.log(4 / 3) + 0.25 * math.log(4), math.inf, 0])
