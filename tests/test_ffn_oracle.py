"""The 64-bit definitions of the 4-bit linear and the gated block, held against hand-worked numbers,
scalar loops and differences (CPU)."""
import math

import numpy as np
import pytest

from oracle import ffn_oracle as O


def test_int4_unpack_and_dequant_by_hand():
    w = np.array([[0x21, 0xF3]], np.uint8)  # low nibble first: 1, 2, 3, 15
    assert O.int4_unpack(w, 4).tolist() == [[1, 2, 3, 15]]
    s = np.array([[0.5, 2.0]])
    assert O.int4_dequant(w, s, None, 4, 2).tolist() == [[-3.5, -3.0, -10.0, 14.0]]
    z = np.array([[1, 15]], np.uint8)
    assert O.int4_dequant(w, s, z, 4, 2).tolist() == [[0.0, 0.5, -24.0, 0.0]]


def test_int4_short_last_group():
    w = np.full((1, 3), 0x99, np.uint8)
    s = np.array([[1.0, 10.0]])
    assert O.int4_dequant(w, s, None, 6, 4).tolist() == [[1, 1, 1, 1, 10, 10]]


@pytest.mark.parametrize("g,u,alpha,limit", [(0.3, -2.0, 1.0, math.inf), (5.0, 3.0, 1.0, 2.0), (-4.0, -9.0, 1.7, 7.0),
                                             (0.0, 0.0, 1.0, math.inf), (-200.0, 1.0, 1.0, math.inf)])
def test_gated_scalar(g, u, alpha, limit):
    t = alpha * min(g, limit)
    want = t * (0.0 if t < -700 else 1.0 / (1.0 + math.exp(-t))) * max(-limit, min(limit, u))
    assert math.isclose(float(O.gated(np.float64(g), np.float64(u), alpha, limit)), want, rel_tol=1e-14, abs_tol=1e-300)


def test_checkpoint_by_hand():
    v = np.zeros((2, 130))
    v[0, :3] = [127.0, -63.5, 0.5]     # scale 1: -63.5 -> -64 (even), 0.5 -> 0
    v[0, 128:] = [2.54, -1.27]         # scale 0.02
    codes, scale = O.checkpoint_int8(v)
    assert codes[0, :3].tolist() == [127, -64, 0]
    assert codes[0, 128:].tolist() == [127, -64]  # -63.5 -> -64
    assert scale[0].tolist() == [1.0, 2.54 / 127] and scale[1].tolist() == [0.0, 0.0]
    assert np.all(codes[1] == 0)
    assert O.checkpoint_values(codes, scale)[0, 128] == 127 * (2.54 / 127)


@pytest.mark.parametrize("alpha,limit", [(1.0, np.inf), (1.3, 0.8)])
def test_backward_is_the_forwards_derivative(alpha, limit):
    r = np.random.default_rng(3)
    M, H, I = 5, 6, 7
    x, w, dh = r.normal(size=(M, H)), r.normal(size=(2 * I, H)), r.normal(size=(M, I))

    def loss(x, w):
        gu = x @ w.T
        return float(np.sum(dh * O.gated(gu[:, :I], gu[:, I:], alpha, limit)))

    gu = x @ w.T
    dx, dw, _ = O.backward(dh, x, w, gu[:, :I], gu[:, I:], alpha, limit)
    e = 1e-6
    for got, arr, other in ((dx, x, lambda a: loss(a, w)), (dw, w, lambda a: loss(x, a))):
        for idx in np.ndindex(arr.shape):
            p, m = arr.copy(), arr.copy()
            p[idx] += e
            m[idx] -= e
            # central difference: O(e^2) third-derivative term plus 2^-52 |loss| / e
            assert abs(got[idx] - (other(p) - other(m)) / (2 * e)) < 1e-7 * (1 + abs(got[idx]))
