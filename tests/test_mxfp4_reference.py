"""The plain MXFP4 and expert-layer implementations of the tests, pinned on hand-computed values (CPU)."""
import numpy as np
import pytest

import mx_reference as R


def test_decode_hand_values():
    # bytes: 0x21 -> codes 1, 2 = 0.5, 1; 0xF7 -> 7, 15 = 6, -6; 0x98 -> 8, 9 = -0, -0.5
    got = R.decode_codes(np.array([[0x21, 0xF7, 0x98, 0x35, 0x64]], np.uint8))[0]
    assert got.tolist() == [0.5, 1.0, 6.0, -6.0, -0.0, -0.5, 3.0, 1.5, 2.0, 4.0]
    assert np.signbit(got[4])


def test_scale_bytes():
    codes = np.full((1, 16), 0x22, np.uint8)  # ones
    for s, want in ((0, 2.0 ** -127), (1, 2.0 ** -126), (127, 1.0), (128, 2.0), (254, 2.0 ** 127)):
        assert (R.decode(codes, np.array([[s]], np.uint8)) == want).all()
    assert np.isnan(R.decode(codes, np.array([[255]], np.uint8))).all()


@pytest.mark.parametrize("v,code", [
    (0.25, 0), (0.2500001, 1), (0.75, 2), (0.7499, 1), (1.25, 2), (1.75, 4), (2.5, 4), (2.51, 5), (3.5, 6), (5.0, 6),
    (5.01, 7), (6.0, 7), (7.99, 7), (-0.0, 8), (-0.25, 8), (-3.5, 14)])
def test_encode_rounds_ties_to_the_even_code(v, code):
    x = np.zeros((1, 32))
    x[0, 0] = 4.0  # largest magnitude 4: scale 2^0
    x[0, 3] = v
    codes, scales = R.encode(x)
    if abs(v) < 8:
        assert scales[0, 0] == 127 and codes[0, 1] >> 4 == code and codes[0, 0] & 15 == 6


def test_encode_scale_of_powers_zeros_and_non_finite():
    x = np.zeros((6, 32))
    x[0, 5] = 2.0 ** 10
    x[1, 5] = 2.0 ** 10 * 1.999
    x[2, 5] = 2.0 ** -126
    x[3, 5] = np.inf
    x[4, 5] = np.nan
    codes, scales = R.encode(x)
    assert scales[:, 0].tolist() == [127 + 8, 127 + 8, 0, 255, 255, 0]
    assert codes[0, 2] >> 4 == 6 and codes[1, 2] >> 4 == 7  # 4; 7.996 -> 6
    assert (codes[3:] == 0).all()


def test_round_trip_of_representable_values():
    rng = np.random.default_rng(0)
    codes = rng.integers(0, 256, (5, 64), np.uint8)
    codes[:, ::16] = (codes[:, ::16] & 0xF0) | 6  # a magnitude of 4 in every block: the same scale comes back
    scales = rng.integers(1, 250, (5, 4), np.uint8)
    c2, s2 = R.encode(R.decode(codes, scales))
    assert (s2 == scales).all() and (c2 == codes).all()


def test_route_ties_masks_and_rows_with_nothing():
    inf = np.inf
    l = np.array([[1.0, 2.0, 2.0, 0.0], [-inf, -inf, -inf, -inf], [-inf, 3.0, -inf, -inf], [0.0, np.nan, 0.0, 0.0],
                  [0.0, inf, 0.0, 0.0]])
    r = R.route(l, 2, True, 1.0)
    assert r[0].tolist() == [0.0, 0.5, 0.5, 0.0]
    assert (r[1] == 0).all() and r[2].tolist() == [0.0, 1.0, 0.0, 0.0]
    assert np.isnan(r[3]).all() and np.isnan(r[4]).all()
    one = R.route(l[:1], 1, True, 1.0)
    assert one[0].tolist() == [0.0, 1.0, 0.0, 0.0]  # the lower index of the two equals


def test_moe_against_a_loop_over_slots():
    rng = np.random.default_rng(1)
    T, E, I, H, k = 3, 4, 6, 5, 2
    x, g, u, d = (rng.standard_normal(s) for s in ((T, H), (E, I, H), (E, I, H), (E, H, I)))
    l = rng.standard_normal((T, E))
    y, _ = R.moe(x, g, u, d, (abs(g), abs(u), abs(d)), l, k, renorm=False, scale=2.0)
    for t in range(T):
        p = np.exp(l[t]) / np.exp(l[t]).sum()
        want = 0
        for e in np.argsort(-l[t])[:k]:
            a = g[e] @ x[t]
            want = want + 2.0 * p[e] * (d[e] @ (a / (1 + np.exp(-a)) * (u[e] @ x[t])))
        assert np.allclose(y[t], want, rtol=1e-12, atol=1e-12)
