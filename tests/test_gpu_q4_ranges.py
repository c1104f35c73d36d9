"""Products with 4-bit weights at the ends of the types' ranges, the few rows' kernel and the tiles alike, against
the fp64 oracle.  Tolerances: test_gpu_q4.py's, (K + groups + 3) 2^-24 of the sum of the terms' magnitudes (3 K
terms where fp32 rows go in three parts) and half a step of the type."""
import numpy as np
import pytest
import torch

from implicit_attribute_decode_amd import ia
from implicit_attribute_decode_amd.pipeline import _DTYPES, Q4Tensor, q4_linear, q4_quantize

from gpu_util import cuda, host
from test_gpu_q4 import TYPES, _assert_linear, _f64, _matrix, _values, ids

pytestmark = pytest.mark.gpu

SIZES = [(1, 50), (17, 50), (40, 50), (5, 16400), (2100, 1100)]  # the last one in tiles
GROUPS = 9


def _weights(rng, N, scales, zeros=None, group=64):
    codes = torch.as_tensor(rng.integers(0, 256, (N, GROUPS * group // 2)).astype(np.uint8), device="cuda")
    zeros = cuda(rng.integers(0, 16, (N, GROUPS))) if zeros is None else zeros
    return Q4Tensor.from_parts(codes, cuda(np.broadcast_to(scales, (N, GROUPS)).astype(np.float32)), zeros, GROUPS * group, group)


def _takes_tiles(M, K, N, dtype):
    return ia.ia_q4_linear_workspace_size(_DTYPES[dtype], M, K, N) > 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=ids)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,N", SIZES)
def test_inputs_near_the_largest_float(M, N, group, dtype):
    """Inputs of 3e38 against weights of a hundredth: a group's inputs times whole numbers pass fp32's range, its sum does
    not (at most 0.15 (3 * 3e38 + 1152 * 1e36) = 3.1e38)."""
    rng = np.random.default_rng(M + N)
    w = _weights(rng, N, rng.uniform(0.001, 0.01, (N, GROUPS)) * np.sign(rng.normal(size=(N, GROUPS))), group=group)
    x = torch.as_tensor(rng.uniform(-1, 1, (M, GROUPS * group)), device="cuda") * 1e36
    x[:, 3], x[:, GROUPS * group // 2], x[:, -1] = 3e38, -3e38, 3e38
    x = x.to(dtype)
    assert M < 1000 or _takes_tiles(M, GROUPS * group, N, dtype)
    y = q4_linear(x, w)
    assert torch.isfinite(y).all()
    _assert_linear(y[-60:], _f64(x)[-60:], _values(w))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=ids)
@pytest.mark.parametrize("M,N", SIZES)
@pytest.mark.parametrize("weights", [2.0 ** 40, 1.0])
def test_inputs_near_the_least_float(M, N, weights, dtype):
    """Inputs of 2^-122 and less down to subnormal ones."""
    rng = np.random.default_rng(M + N)
    w = _weights(rng, N, rng.uniform(0.1, 1, (N, GROUPS)) * weights)
    x = (_matrix(rng, M, GROUPS * 64) * 2.0 ** -122).to(dtype)
    x[:, :8] *= 2.0 ** -6
    y, v, rows = q4_linear(x, w)[-60:], _values(w), _f64(x)[-60:]
    if dtype == torch.float32:
        _assert_linear(y, rows, v)
    else:  # bf16 inputs are taken whole: what is below fp32's least value is lost, half of 2^-149 a term
        want, size = rows @ v.T, np.abs(rows) @ np.abs(v).T
        tol = (v.shape[1] + 22) * (2.0 ** -24 * size + 2.0 ** -150) + 2.0 ** -8 * np.abs(want) * (1 + 2.0 ** -10) + 2.0 ** -134
        assert (np.abs(_f64(y) - want) <= tol).all()


@pytest.mark.parametrize("M,N", SIZES)
def test_scales_past_2_64(M, N):
    """The largest scales over inputs of a size that keeps the results below fp32's end; zeros elsewhere."""
    rng = np.random.default_rng(M + N)
    scales = rng.uniform(0.5, 1, (N, GROUPS)) * 2.0 ** rng.integers(60, 124, (N, GROUPS))
    w = _weights(rng, N, scales)
    x = _matrix(rng, M, GROUPS * 64) * 2.0 ** -20
    y = q4_linear(x, w)
    assert torch.isfinite(y).all()
    _assert_linear(y[-60:], _f64(x)[-60:], _values(w))
    assert (q4_linear(torch.zeros_like(x), w) == 0).all()


@pytest.mark.parametrize("tiny", [2.0 ** -100, -2.0 ** -81, 2.0 ** -79, 2.0 ** -66, -2.0 ** -60, 0.0])
@pytest.mark.parametrize("M,N", SIZES)
def test_large_sums_that_cancel(M, N, tiny):
    """A group of scale 2^42, one of next to nothing and one of -2^42 over the same codes and inputs: whole numbers, whose
    sums (64 * 15 * 3 * 2^42 at most) are exact and cancel, so that the other groups' sum remains as if alone."""
    rng = np.random.default_rng(M + N)
    scales = rng.uniform(0.001, 0.01, (N, GROUPS))
    scales[:, 0], scales[:, 1], scales[:, 2] = 2.0 ** 42, tiny, -2.0 ** 42
    codes = rng.integers(0, 256, (N, GROUPS * 32)).astype(np.uint8)
    codes[:, 64:96] = codes[:, :32]
    w = Q4Tensor.from_parts(torch.as_tensor(codes, device="cuda"), cuda(scales.astype(np.float32)), 3, GROUPS * 64, 64)
    x = _matrix(rng, M, GROUPS * 64, torch.float16)
    x[:, :192] = torch.as_tensor(rng.integers(-3, 4, (M, 192)), device="cuda")
    x[:, 128:192] = x[:, :64]
    assert M < 1000 or _takes_tiles(M, GROUPS * 64, N, torch.float16)
    y = q4_linear(x, w)
    # what the tiny scale adds is below 2^-60 * 64 * 12 * 3
    _assert_linear(y[-60:], _f64(x[-60:, 192:]), _values(w)[:, 192:])


@pytest.mark.parametrize("power", [-30, -25, -24, -23, -18, -14, -10, 0, 7, 8, 9, 12])
@pytest.mark.parametrize("M,N", SIZES)
def test_fp16_scales_of_every_power(M, N, power):
    """Scales about 2^power, over inputs of a size that keeps the results in fp16's middle."""
    rng = np.random.default_rng(M + N)
    w = _weights(rng, N, rng.uniform(1, 2, (N, GROUPS)) * 2.0 ** power * np.sign(rng.normal(size=(N, GROUPS))))
    x = (torch.as_tensor(rng.uniform(-1, 1, (M, GROUPS * 64)), device="cuda") * 2.0 ** min(max(-power, -12), 15)).half()
    y = q4_linear(x, w)
    assert torch.isfinite(y).all() and (y != 0).any()
    _assert_linear(y[-60:], _f64(x)[-60:], _values(w))


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("M,N", SIZES)
def test_infinite_inputs_over_scales_of_any_size(M, N, dtype):
    """An infinite input gives an infinity of the weight's sign however small the scale, NaN against a weight of zero (of a
    zero scale as well)."""
    rng = np.random.default_rng(M + N)
    scales = rng.uniform(0.001, 0.01, (N, GROUPS))
    scales[:, 1], scales[:, 3], scales[:, 4], scales[:, 6], scales[:, 7] = 2.0 ** -100, -2.0 ** -81, 2.0 ** -66, 0.0, 2.0 ** -40
    w = _weights(rng, N, scales)
    v = _values(w)
    for g in range(GROUPS):
        x = _matrix(rng, M, GROUPS * 64, dtype)
        k = 64 * g + int(rng.integers(64))
        x[M - 1, k] = float("inf") * (1 if g % 2 else -1)
        y = _f64(q4_linear(x, w))
        assert np.isfinite(y[:M - 1]).all()
        zero = v[:, k] == 0
        assert np.isnan(y[M - 1, zero]).all() and zero.all() == (g == 6)
        assert np.array_equal(y[M - 1, ~zero], (1 if g % 2 else -1) * np.sign(v[~zero, k]) * np.inf)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("M,N", SIZES)
def test_weights_of_the_whole_range(M, N, dtype):
    """Weights of either sign up to the largest float: their scales pass 2^125, their values (from the rounding of the zero)
    fp32's range, and a code less its zero, -8, times 2^125 does so too.  Small inputs and zeros give the products of those values all the same."""
    rng = np.random.default_rng(M + N)
    wf = rng.normal(size=(N, GROUPS * 64))
    big = float(np.finfo(np.float32).max)
    wf[:, 5], wf[:, 9], wf[:, 200], wf[:, 250], wf[:, 400], wf[:, 440] = -3.3e38, 3.13e38, -big, 0.3 * big, big, -big
    w = q4_quantize(torch.as_tensor(wf, device="cuda").float(), 64)
    v = _values(w)
    assert np.abs(v).max() > big and float(w.scales[:, 0].min()) > 2.0 ** 125 and int(w.zeros[0, 0]) == 8
    x = _matrix(rng, M, GROUPS * 64, dtype)
    x[:, :64] = x[:, 192:256] = x[:, 384:448] = 0
    y = q4_linear(x, w)
    assert torch.isfinite(y).all()
    _assert_linear(y[-60:], _f64(x)[-60:], v)
    if dtype != torch.float16:
        x = x * 2.0 ** -20
        x[:, :64] = x[:, 192:256] = x[:, 384:448] = 2.0 ** -30
        y = q4_linear(x, w)
        assert torch.isfinite(y).all()
        _assert_linear(y[-60:], _f64(x)[-60:], v)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,K,N", [(1, 1030, 8192), (1, 1030, 8193), (16, 300, 8200), (3, 4096, 12289)])
def test_few_rows_of_wide_layers(M, K, N, group, dtype):
    """Either side of the number of outputs from which a wave takes two tiles of them."""
    rng = np.random.default_rng(M + K + N)
    x, w = _matrix(rng, M, K, dtype), q4_quantize(_matrix(rng, N, K, scale=K ** -0.5), group)
    bias = cuda(rng.normal(size=N).astype(np.float32))
    _assert_linear(q4_linear(x, w, bias, "relu"), _f64(x), _values(w), _f64(bias), relu=True)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("M,K,N", [(20, 2 ** 20 - 5, 60), (20, 2 ** 20 + 3, 60), (3, 2 ** 20 + 3, 60), (20, 2 ** 22 + 70, 5)])
def test_a_million_inputs(M, K, N, dtype):
    """Around the inputs up to which tiles are taken: whole numbers, whose sums (2^22 * 15 at most) fp32 holds up to 2^24,
    which sums of inputs -1, 0 and 1 at random do not reach (the oracle says so), so that they are exact."""
    rng = np.random.default_rng(K + M)
    groups = -(-K // 128)
    codes = rng.integers(0, 256, (N, groups * 64)).astype(np.uint8)
    w = Q4Tensor.from_parts(torch.as_tensor(codes, device="cuda"), torch.ones((N, groups), device="cuda"), 7, K, 128)
    x = rng.integers(-1, 2, (M, K)).astype(np.float32)
    v = _values(w).astype(np.float32)
    want = x.astype(np.float64) @ v.astype(np.float64).T
    assert np.abs(want).max() < 60000
    got = q4_linear(cuda(x).to(dtype), w)
    assert torch.equal(got.cpu(), torch.as_tensor(want).to(dtype))
