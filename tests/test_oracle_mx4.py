"""Pins of the MXFP4 oracle (oracle/mx4.py) against what the format fixes:
every code, the rounding's decision points, the scale's exponent, and the
gradients of a layer whose operands the format holds exactly."""
import numpy as np

from oracle import mx4 as O
from oracle import train as T


def test_every_code_and_scale_reads_back():
    for byte in (0, 1, 100, 127, 200, 254):
        codes = np.arange(16, dtype=np.uint8)
        c = np.tile(codes[0::2] | (codes[1::2] << 4), 2)[None]
        v = O.dequantize(c, np.array([[byte]], np.uint8), 32)[0]
        want = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6]) * 2.0 ** (byte - 127)
        assert np.array_equal(v[:8], want) and np.array_equal(v[8:16], -want)
    assert np.isnan(O.dequantize(c, np.array([[255]], np.uint8), 32)).all()


def test_decision_points_round_to_the_even_code():
    # with 4 in the block its scale is 1
    x = np.array([[4, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 7.9, -0.25, -5, 0.2500001, 0.7499999, 5.0001, -0.0]])
    want = [4, 0, 1, 1, 2, 2, 4, 4, 6, -0.0, -4, 0.5, 0.5, 6, -0.0]
    got = O.values(x)[0]
    assert np.array_equal(got, want) and np.array_equal(np.signbit(got), np.signbit(want))


def test_scale_is_the_exponent_of_the_largest_value_minus_two():
    for m, byte in ((1.0, 125), (1.9999, 125), (2.0, 126), (6.0, 127), (2.0 ** -126, 0), (2.0 ** -125, 0),
                    (2.0 ** -124, 1), (3e38, 252), (2.0 ** -149, 0), (0.0, 0)):
        assert O.quantize(np.array([[m, m / 3]]))[1][0, 0] == byte, m
    assert O.quantize(np.array([[1.0, np.nan]]))[1][0, 0] == 255
    assert O.quantize(np.array([[1.0, -np.inf]]))[1][0, 0] == 255


def test_error_bound_and_idempotence():
    rng = np.random.default_rng(1)
    x = rng.normal(0, 1, (50, 70)) * np.exp(rng.normal(0, 4, (50, 1)))
    q = O.values(x)
    pad = np.zeros((50, 96))
    pad[:, :70] = np.abs(x)
    m = pad.reshape(50, 3, 32).max(-1).repeat(32, 1)[:, :70]
    scale = 2.0 ** (np.floor(np.log2(m)) - 2)
    # half the widest step, or the cut from just below 8 to 6
    assert np.all(np.abs(q - x) <= 2 * scale) and np.all(np.abs(q - x)[np.abs(x) < 6 * scale] <= 1.0 * scale.max())
    assert np.array_equal(O.values(q), q)


def test_layer_gradients_of_exact_operands_match_differences():
    """Matrices of E2M1 values are exact in every block: the layer is linear
    and its central differences are its gradients."""
    rng = np.random.default_rng(2)
    grid = np.concatenate([O.GRID[1:], -O.GRID[1:]])
    x, w, dy = (rng.choice(grid, s) for s in ((5, 40), (7, 40), (5, 7)))
    g = O.linear_backward(dy, x, w)
    loss = lambda a, b: (dy * O.product(a, b)[0]).sum()  # noqa: E731
    for (i, j) in ((0, 0), (4, 39), (2, 33)):
        d = np.zeros_like(x)
        d[i, j] = 0.5
        assert np.isclose(loss(x + d, w) - loss(x - d, w), g["x"][0][i, j], rtol=1e-13)
        d = np.zeros_like(w)
        d[i, j] = 0.5
        assert np.isclose(loss(x, w + d) - loss(x, w - d), g["weight"][0][i, j], rtol=1e-13)


def test_clip_factor():
    assert T.clip_factor([np.array([3.0]), np.array([[4.0]])], 10.0) == (5.0, 1.0)
    assert T.clip_factor([np.array([3.0]), np.array([[4.0]])], 1.0) == (5.0, 0.2)
    assert T.clip_factor([], 1.0) == (0.0, 1.0)
