"""MXFP4 quantisation, read-back, products and the layer's gradients through
the C ABI against the fp64 oracle.

Codes, scales and read-back values are fixed by the format: compared exactly.
A product of n terms accumulated in fp32 is within n 2^-24 of the sum of its
terms' magnitudes (plus the bias and a margin of 2 operations), then rounded
once to its type (2^-24, 2^-11, 2^-8, half the smallest subnormal)."""
import numpy as np
import pytest
import torch

from oracle import mx4 as O
from implicit_attribute_decode_amd import ia
from implicit_attribute_decode_amd.pipeline import (Mx4Linear, Mx4Tensor, mx4_linear, mx4_linear_backward, mx4_matmul,
                                                    mx4_quantize)

from gpu_util import cuda, host

pytestmark = pytest.mark.gpu

UNIT = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -150, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}
TYPES = list(UNIT)
ids = lambda v: str(v).replace("torch.", "") if isinstance(v, torch.dtype) else None  # noqa: E731


def _f64(t):
    return t.double().cpu().numpy()


def _matrix(rng, rows, cols, dtype=torch.float32, scale=1.0):
    x = rng.normal(0, scale, (rows, cols)) * np.exp(rng.normal(0, 0.7, (rows, 1)))
    return torch.as_tensor(x.astype(np.float32), device="cuda").to(dtype)


def _assert_quantized(q: Mx4Tensor, x):
    codes, scales = O.quantize(x)
    assert np.array_equal(host(q.scales), scales)
    assert np.array_equal(host(q.codes), codes)


def _assert_near(got, want, scale, terms, dtype):
    """got (a tensor of dtype) against want with the error of `terms` fp32 operations on `scale`."""
    g = _f64(got)
    assert np.array_equal(np.isnan(g), np.isnan(want))
    ok = ~np.isnan(want)
    tol = (terms + 3) * 2.0 ** -24 * scale + UNIT[dtype] * np.abs(want) * (1 + 2.0 ** -10) + TINY[dtype]
    assert np.all(np.abs(g - want)[ok] <= tol[ok]), float((np.abs(g - want) / tol)[ok].max())


SHAPES = [(1, 1), (1, 31), (3, 32), (5, 33), (64, 64), (2, 1000), (129, 250), (33, 96), (300, 7), (1000, 160), (31, 4099)]


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_quantize_and_read_back(rows, cols, dtype):
    x = _matrix(np.random.default_rng(rows * cols), rows, cols, dtype)
    q, t = mx4_quantize(x), mx4_quantize(x, transpose=True)
    _assert_quantized(q, _f64(x))
    _assert_quantized(t, _f64(x).T)
    for out in TYPES:
        want = torch.as_tensor(O.values(_f64(x))).to(out)  # one rounding from 64 bits
        assert torch.equal(q.dequantize(out).cpu(), want)
        assert torch.equal(t.dequantize(out).cpu(), torch.as_tensor(O.values(_f64(x).T)).to(out))


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
def test_quantize_decision_points_and_extremes(dtype):
    """Ties, zeros of both signs, subnormal and largest values, blocks of zeros."""
    base = np.array([4, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 6, 7, 7.5, -0.25, -0.75, -5, 0.0, -0.0, 0.26, 0.24, 0.74,
                     0.76, 1.24, 1.26, 1.74, 1.76, 2.49, 2.51, 3.49, 3.51, 4.99, 5.01, 1e-3, -1e-3])
    top = {torch.float32: 125, torch.float16: 13, torch.bfloat16: 125}[dtype]
    low = {torch.float32: -149, torch.float16: -24, torch.bfloat16: -133}[dtype]
    rows = [base * 2.0 ** e for e in (0, 1, -3, top, top - 1, low, low + 2, low + 5, -124, -125, -126, -127, -128)]
    rows += [np.zeros(32), -np.zeros(32), np.full(32, 2.0 ** low), np.full(32, torch.finfo(dtype).max)]
    x = torch.as_tensor(np.array(rows), device="cuda").to(dtype)
    q = mx4_quantize(x)
    _assert_quantized(q, _f64(x))
    _assert_quantized(mx4_quantize(x.t().contiguous(), transpose=True), _f64(x))
    got = q.dequantize(torch.float32)
    want = torch.as_tensor(O.values(_f64(x))).float()
    assert torch.equal(got.cpu(), want) and torch.equal(torch.signbit(got).cpu(), torch.signbit(want))


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_blocks_that_are_not_finite(dtype, bad):
    rng = np.random.default_rng(4)
    x = _matrix(rng, 20, 150, dtype)
    x[3, 40] = x[7, 149] = x[19, 0] = bad
    q = mx4_quantize(x)
    _assert_quantized(q, _f64(x))
    _assert_quantized(mx4_quantize(x, transpose=True), _f64(x).T)
    v = host(q.dequantize())
    assert np.isnan(v[3, 32:64]).all() and np.isnan(v[7, 128:]).all() and np.isnan(v).sum() == 32 + 22 + 32
    w = _matrix(rng, 30, 150)
    y = mx4_linear(x, mx4_quantize(w), act="relu")
    assert torch.isnan(y[[3, 7, 19]]).all() and int(torch.isnan(y).sum()) == 3 * 30
    c = mx4_matmul(mx4_quantize(w), q)
    assert torch.isnan(c[:, [3, 7, 19]]).all() and int(torch.isnan(c).sum()) == 3 * 30


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
def test_quantize_rows_of_wider_arrays_and_repeated_rows(dtype):
    rng = np.random.default_rng(5)
    wide = _matrix(rng, 70, 203, dtype)
    for view in (wide[:, 1:100], wide[3:40, 64:192], wide[::2, 5:69], wide[:, 7:8], wide[5:6, 2:]):
        _assert_quantized(mx4_quantize(view), _f64(view))
        _assert_quantized(mx4_quantize(view, transpose=True), _f64(view).T)
    row = wide[9:10, 3:90].expand(50, 87)
    _assert_quantized(mx4_quantize(row), _f64(row))
    _assert_quantized(mx4_quantize(row, transpose=True), _f64(row).T)
    q = mx4_quantize(wide)
    out = torch.full((70, 300), 5.0, device="cuda", dtype=dtype)
    q.dequantize(out=out[:, 11:214])
    assert torch.equal(out[:, 11:214], q.dequantize(dtype))
    assert (out[:, :11] == 5).all() and (out[:, 214:] == 5).all()


def test_empty_matrices():
    for rows, cols in ((0, 5), (5, 0), (0, 0)):
        x = torch.empty((rows, cols), device="cuda")
        for t in (False, True):
            q = mx4_quantize(x, transpose=t)
            assert tuple(q.dequantize().shape) == ((cols, rows) if t else (rows, cols))
    b = torch.tensor([1.0, -2.0], device="cuda")
    none = mx4_quantize(torch.empty((2, 0), device="cuda"))
    y = mx4_linear(torch.empty((3, 0), device="cuda"), none, b, "relu")
    assert host(y).tolist() == [[1.0, 0.0]] * 3
    assert tuple(mx4_linear(torch.empty((0, 40), device="cuda"), mx4_quantize(torch.ones((6, 40), device="cuda"))).shape) == (0, 6)
    w = torch.ones((6, 40), device="cuda")
    g = mx4_linear_backward(torch.empty((0, 6), device="cuda"), torch.empty((0, 40), device="cuda"),
                            mx4_quantize(w, transpose=True))
    assert tuple(g["x"].shape) == (0, 40) and (g["weight"] == 0).all() and (g["bias"] == 0).all()


PRODUCTS = [(1, 1, 1), (1, 70, 33), (2, 300, 4096), (5, 7, 31), (16, 16, 32), (17, 58, 192), (64, 64, 64),
            (129, 130, 250), (300, 256, 256), (33, 11, 64), (257, 65, 129), (8, 1000, 2000), (70, 515, 160),
            (500, 300, 1024), (1030, 520, 416)]


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_matmul(M, N, K, dtype):
    rng = np.random.default_rng(M + N + K)
    a, b = _matrix(rng, M, K), _matrix(rng, N, K)
    bias = _matrix(rng, 1, N)[0]
    qa, qb = mx4_quantize(a), mx4_quantize(b)
    va, vb = O.values(_f64(a)), O.values(_f64(b))
    for bi, act in ((None, "none"), (bias, "relu")):
        want, scale = O.product(va, vb, None if bi is None else _f64(bi), act == "relu")
        got = mx4_matmul(qa, qb, bi, act, dtype)
        _assert_near(got, want, scale, K, dtype)
        assert torch.equal(got, mx4_matmul(qa, qb, bi, act, dtype))


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("M,N,K", [(3900, 4087, 2999), (4090, 3850, 4800)])
def test_matmul_of_many_long_rows(M, N, K, dtype):
    rng = np.random.default_rng(M + N + K)
    a, b, bias = _matrix(rng, M, K), _matrix(rng, N, K), _matrix(rng, 1, N)[0]
    want, scale = O.product(O.values(_f64(a)), O.values(_f64(b)), _f64(bias), True)
    _assert_near(mx4_matmul(mx4_quantize(a), mx4_quantize(b), bias, "relu", dtype), want, scale, K, dtype)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_linear(M, N, K, dtype):
    rng = np.random.default_rng(M * N + K)
    x, w = _matrix(rng, M, K, dtype), _matrix(rng, N, K)
    bias = _matrix(rng, 1, N)[0]
    q = mx4_quantize(w)
    for bi, act in ((None, "relu"), (bias, "none")):
        want, scale = O.linear(_f64(x), _f64(w), None if bi is None else _f64(bi), act == "relu")
        got = mx4_linear(x, q, bi, act)
        _assert_near(got, want, scale, K, dtype)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
def test_linear_strided_repeated_and_into_wider_outputs(dtype):
    rng = np.random.default_rng(6)
    for M, N, K in ((77, 58, 192), (3, 90, 70), (200, 300, 65)):
        wide = _matrix(rng, M, K + 37, dtype)
        q = mx4_quantize(_matrix(rng, N, K))
        for x in (wide[:, 5:5 + K], wide[:, 8:8 + K], wide[::2, :K], wide[1:2, 3:3 + K].expand(M, K)):
            out = torch.full((x.shape[0], N + 9), 3.0, device="cuda", dtype=dtype)
            want = mx4_linear(x.contiguous(), q, act="relu")
            assert torch.equal(mx4_linear(x, q, act="relu"), want)
            mx4_linear(x, q, act="relu", out=out[:, 4:4 + N])
            assert torch.equal(out[:, 4:4 + N], want) and (out[:, :4] == 3).all() and (out[:, 4 + N:] == 3).all()


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("M,N,K", [(1, 50, 16_000), (4, 2100, 8192), (20, 33, 3999), (64, 40, 2017), (64, 256, 8190),
                                   (1, 16, 30_001), (3, 20_000, 100)])
def test_linear_of_few_rows(M, N, K, dtype):
    rng = np.random.default_rng(M + N + K)
    x, w, bias = _matrix(rng, M, K + 3, dtype)[:, 3:], _matrix(rng, N, K), _matrix(rng, 1, N)[0]
    want, scale = O.linear(_f64(x), _f64(w), _f64(bias), True)
    _assert_near(mx4_linear(x, mx4_quantize(w), bias, "relu"), want, scale, K, dtype)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("M,N,K", [(65, 513, 256), (300, 1100, 31), (1000, 2304, 200)])
def test_linear_of_few_inputs_and_many_outputs(M, N, K, dtype):
    rng = np.random.default_rng(M + N * K)
    x, w, bias = _matrix(rng, M, K, dtype), _matrix(rng, N, K), _matrix(rng, 1, N)[0]
    want, scale = O.linear(_f64(x), _f64(w), _f64(bias), True)
    wide = torch.full((M, N + 24), 3.0, device="cuda", dtype=dtype)
    for first in (0, 8, 11):
        out = wide[:, first:first + N]
        mx4_linear(x, mx4_quantize(w), bias, "relu", out=out)
        _assert_near(out, want, scale, K, dtype)
        assert (wide[:, :first] == 3).all() and (wide[:, first + N:] == 3).all()
        wide.fill_(3.0)
    dy = _matrix(rng, M, K, dtype, 1e-2)  # the layer back: K outputs of N inputs
    back = mx4_linear_backward(dy, wide[:, :N], mx4_quantize(w))["x"]
    _assert_near(back, *O.linear_backward(_f64(dy), _f64(wide[:, :N]), _f64(w).T)["x"], K, dtype)


BACKWARD = [(1, 1, 1), (3, 5, 7), (31, 32, 33), (64, 58, 192), (200, 256, 192), (129, 11, 64), (1000, 56, 32),
            (4099, 58, 250), (33, 300, 70), (260, 515, 300), (20_003, 64, 64)]


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("M,N,K", BACKWARD)
@pytest.mark.parametrize("relu", [False, True])
def test_linear_backward(M, N, K, dtype, relu):
    rng = np.random.default_rng(M + 2 * N + 3 * K + relu)
    x, w, dy = _matrix(rng, M, K, dtype), _matrix(rng, N, K), _matrix(rng, M, N, dtype, 1e-2)
    y = torch.relu(_matrix(rng, M, N, dtype)) if relu else None
    want = O.linear_backward(_f64(dy), _f64(x), _f64(w), None if y is None else _f64(y))
    wt = mx4_quantize(w, transpose=True)
    got = mx4_linear_backward(dy, x, wt, y)
    _assert_near(got["x"], *want["x"], N, dtype)
    _assert_near(got["weight"], *want["weight"], M, torch.float32)
    _assert_near(got["bias"], *want["bias"], M, torch.float32)
    again = mx4_linear_backward(dy, x, wt, y)
    assert all(torch.equal(got[k], again[k]) for k in got)
    part = mx4_linear_backward(dy, x, None, y, want_x=False)
    assert part["x"] is None and torch.equal(part["weight"], got["weight"]) and torch.equal(part["bias"], got["bias"])


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
def test_backward_of_strided_and_broadcast_gradients(dtype):
    """Upstream gradients that are rows of a wider array, or one row repeated (a sum's gradient)."""
    rng = np.random.default_rng(7)
    M, N, K = 150, 58, 70
    xw, dw, yw = _matrix(rng, M, K + 11, dtype), _matrix(rng, M, N + 5, dtype), _matrix(rng, M, N + 3, dtype)
    wt = mx4_quantize(_matrix(rng, N, K), transpose=True)
    x, y = xw[:, 3:3 + K], yw[:, 1:1 + N]
    for dy in (dw[:, 2:2 + N], dw[4:5, :N].expand(M, N)):
        got = mx4_linear_backward(dy, x, wt, y)
        want = mx4_linear_backward(dy.contiguous(), x.contiguous(), wt, y.contiguous())
        assert all(torch.equal(got[k], want[k]) for k in want)


def test_masked_gradients_that_are_not_finite_do_not_count():
    """dy is NaN or infinite where the ReLU was off: no gradient sees it; y = NaN counts as off."""
    rng = np.random.default_rng(8)
    M, N, K = 70, 40, 50
    x, w, dy = _matrix(rng, M, K), _matrix(rng, N, K), _matrix(rng, M, N)
    y = torch.relu(_matrix(rng, M, N))
    y[5] = float("nan")
    y[6] = 0.0
    off = ~(y > 0)
    bad = torch.where(off, torch.full_like(dy, float("nan")), dy)
    wt = mx4_quantize(w, transpose=True)
    got, want = mx4_linear_backward(bad, x, wt, y), mx4_linear_backward(torch.where(off, 0.0, dy), x, wt)
    for k in want:
        assert torch.equal(got[k], want[k]) and torch.isfinite(got[k]).all()
    assert (got["x"][5:7] == 0).all()  # rows whose mask leaves nothing


@pytest.mark.parametrize("act", ["none", "relu"])
def test_gradients_match_differences(act):
    """Matrices of E2M1 values are exact in every block, so the layer is
    (piecewise) linear and its central differences are its gradients, both
    exact in fp32; biases keep every ReLU away from its corner."""
    rng = np.random.default_rng(9)
    grid = np.concatenate([O.GRID[1:], -O.GRID[1:]])
    M, N, K = 40, 33, 70
    x, w, dy = (rng.choice(grid, s).astype(np.float32) for s in ((M, K), (N, K), (M, N)))
    bias = np.where(np.arange(N) % 3 == 0, -6000.0, 6000.0).astype(np.float32)
    L = Mx4Linear(cuda(w), cuda(bias), act)
    y = L(cuda(x))
    g = {k: _f64(v) for k, v in L.backward(cuda(x), cuda(dy), y).items()}

    def loss(x_, w_, b_):
        return float((_f64(Mx4Linear(cuda(w_), cuda(b_), act)(cuda(x_))) * dy).sum())

    for i, j in ((0, 0), (39, 69), (20, 33), (7, 64)):
        # a step leaves the grid for some values: the entry is moved onto two grid points, one apart
        hi, lo = x.copy(), x.copy()
        hi[i, j], lo[i, j] = 1.5, 0.5
        assert loss(hi, w, bias) - loss(lo, w, bias) == g["x"][i, j]
    for i, j in ((0, 0), (32, 69), (11, 31), (1, 5)):
        hi, lo = w.copy(), w.copy()
        hi[i, j], lo[i, j] = 1.5, 0.5
        assert loss(x, hi, bias) - loss(x, lo, bias) == g["weight"][i, j]
    for i in (0, 1, 32):
        e = np.zeros_like(bias)
        e[i] = 0.5
        assert loss(x, w, bias + e) - loss(x, w, bias - e) == g["bias"][i]


def test_offsets_past_32_bits():
    """Rows and codes beyond 2^32 elements and bytes: the far rows equal the same rows taken alone."""
    rng = np.random.default_rng(10)
    row = (1 << 31) + 8
    far = torch.empty(2 * row + 100, device="cuda", dtype=torch.float16)
    x = far.as_strided((3, 100), (row, 1))
    x.copy_(_matrix(rng, 3, 100, torch.float16))
    q = mx4_quantize(x)
    _assert_quantized(q, _f64(x))
    _assert_quantized(mx4_quantize(x, transpose=True), _f64(x).T)
    far.fill_(0)
    q.dequantize(out=x)
    assert torch.equal(x, q.dequantize(torch.float16))
    del far, x
    M, K = 2_200_000, 4096  # 4.5e9 bytes of codes
    codes = torch.randint(0, 256, (M, K // 2), dtype=torch.uint8, device="cuda")
    scales = torch.randint(120, 130, (M, K // 32), dtype=torch.uint8, device="cuda")
    b = mx4_quantize(_matrix(rng, 5, K))
    c = mx4_matmul(Mx4Tensor(codes, scales, K), b, dtype=torch.float16)
    at = M - 300
    tail = mx4_matmul(Mx4Tensor(codes[at:].clone(), scales[at:].clone(), K), b, dtype=torch.float16)
    want, scale = O.product(O.dequantize(host(codes[at:]), host(scales[at:]), K), _f64(b.dequantize()))
    _assert_near(c[at:], want, scale, K, torch.float16)
    _assert_near(tail, want, scale, K, torch.float16)
    v = Mx4Tensor(codes, scales, K).dequantize(torch.float16)
    assert torch.equal(v[at:], Mx4Tensor(codes[at:].clone(), scales[at:].clone(), K).dequantize(torch.float16))


def test_sums_longer_than_32_bit_offsets_reach():
    """33.5M terms over 130 rows (2.2 GB of codes in one tile's rows): values of
    0.5 and 1 of either sign, so that every partial sum is exact in fp32."""
    rows, K = 130, (1 << 25) + 96
    gen = torch.Generator(device="cuda").manual_seed(3)

    def codes(n):
        pick = torch.tensor([0x11, 0x12, 0x21, 0x22, 0x91, 0x19, 0xa1, 0x1a, 0xaa, 0x99, 0x9a, 0xa9], device="cuda",
                            dtype=torch.uint8)
        # as many of either sign on average: the sums stay small
        return pick[torch.randint(0, 12, (n, K // 2), generator=gen, device="cuda", dtype=torch.int32)]

    a = torch.cat([codes(26) for _ in range(rows // 26)])
    b = codes(3)
    one = lambda n: torch.full((n, K // 32), 127, dtype=torch.uint8, device="cuda")  # noqa: E731
    got = mx4_matmul(Mx4Tensor(a, one(rows), K), Mx4Tensor(b, one(3), K))
    want = torch.zeros((rows, 3), dtype=torch.float64, device="cuda")
    step = 1 << 22
    for k in range(0, K, step):
        n = min(step, K - k)
        part = lambda c, r: Mx4Tensor(c[:, k // 2:(k + n) // 2].contiguous(),  # noqa: E731
                                      torch.full((r, n // 32), 127, dtype=torch.uint8, device="cuda"), n).dequantize()
        want += part(a, rows).double() @ part(b, 3).double().t()
    assert torch.equal(got.double(), want)


def test_backward_of_rows_far_apart():
    """Row strides beyond what the narrow kernels address."""
    rng = np.random.default_rng(12)
    M, N, K, far = 40, 58, 70, (1 << 22) + 8
    dy, x, y = (_matrix(rng, M, c, torch.float16) for c in (N, K, N))
    wt = mx4_quantize(_matrix(rng, N, K), transpose=True)
    want = mx4_linear_backward(dy, x, wt, y)

    def apart(t):
        return torch.empty(M * far, dtype=torch.float16, device="cuda").as_strided(tuple(t.shape), (far, 1)).copy_(t)

    for args in ((apart(dy), x, y), (dy, apart(x), y), (dy, x, apart(y))):
        got = mx4_linear_backward(args[0], args[1], wt, args[2])
        assert torch.equal(got["x"], want["x"])
        for k in ("weight", "bias"):  # another order of summation
            ref, scale = O.linear_backward(_f64(dy), _f64(x), np.zeros((N, K)), _f64(y))[k]
            _assert_near(got[k], ref, scale, M, torch.float32)


def test_side_stream_and_graph_replays():
    """The layer's forward and backward on another stream, and replayed from a graph with eager work between."""
    rng = np.random.default_rng(11)
    M, N, K = 3000, 256, 192
    x, dy = _matrix(rng, M, K, torch.float16), _matrix(rng, M, N, torch.float16)
    L = Mx4Linear(_matrix(rng, N, K), _matrix(rng, 1, N)[0], "relu")
    y = L(x)
    want = {**L.backward(x, dy, y), "y": y}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ys = L(x)
        got = {**L.backward(x, dy, ys), "y": ys}
    torch.cuda.synchronize()
    assert all(torch.equal(got[k], want[k]) for k in want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.update()
        yg = L(x)
        out = {**L.backward(x, dy, yg), "y": yg}
    for _ in range(3):
        for t in out.values():
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out[k], want[k]) for k in want)
        L.backward(_matrix(rng, 500, K), _matrix(rng, 500, N), torch.relu(_matrix(rng, 500, N)))
        torch.cuda.synchronize()


def test_refusals():
    x = torch.ones((4, 64), device="cuda")
    w = mx4_quantize(torch.ones((8, 64), device="cuda"))
    for call in (lambda: mx4_quantize(x.double()), lambda: mx4_quantize(x[:, ::2]), lambda: mx4_quantize(x[0]),
                 lambda: mx4_linear(x[:, :32], w), lambda: mx4_linear(x, w, torch.ones(7, device="cuda")),
                 lambda: mx4_linear(x, w, out=torch.empty((4, 8), device="cuda", dtype=torch.float16)),
                 lambda: mx4_linear_backward(torch.ones((4, 8), device="cuda"), x, w),  # not transposed
                 lambda: mx4_linear_backward(torch.ones((3, 8), device="cuda"), x, None, want_x=False),
                 lambda: Mx4Tensor(w.codes, w.scales, 65), lambda: Mx4Tensor(w.codes.cpu(), w.scales.cpu(), 64),
                 lambda: w.dequantize(out=torch.empty((8, 63), device="cuda")),
                 lambda: Mx4Linear(torch.ones((8, 64), device="cuda"), act="gelu"),
                 lambda: Mx4Linear(torch.ones((8, 64), device="cuda"), act="relu").backward(x, x[:, :8])):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ia.IAError) as e:  # an output of repeated rows
        w.dequantize(out=torch.empty((1, 64), device="cuda").expand(8, 64))
    assert e.value.status == ia.IA_ERR_INVALID_ARG
    with pytest.raises(ia.IAError) as e:
        mx4_matmul(w, mx4_quantize(x[:, :32].contiguous()))
    assert e.value.status == ia.IA_ERR_INVALID_ARG
    n = ia.ia_mx4_linear_backward_workspace_size(4, 8, 64)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    with pytest.raises(ia.IAError) as e:
        ia.ia_mx4_linear_backward(torch.ones((4, 8), device="cuda"), 8, None, 0, x, 64, ia.IA_DTYPE_F32, 4, 8, 64, None,
                                  None, 0, torch.empty((8, 64), device="cuda"), None, ws[: n // 2])
    assert e.value.status == ia.IA_ERR_WORKSPACE_TOO_SMALL
