"""Products with 4-bit weights where they go in tiles of 256 x 256, whole and split over K: which kernel ran is read from
the library's profile, so that these tests say when a change of the choice leaves the wide tiles without one."""
import numpy as np
import pytest
import torch

from implicit_attribute_decode_amd import ia
from implicit_attribute_decode_amd.pipeline import q4_linear, q4_quantize

import test_gpu_q4 as Q
import test_gpu_q4_ranges as R
from gpu_util import cuda, host

pytestmark = pytest.mark.gpu

WIDE, JOIN = "q4_matmul_kernel<256>", "q4_join_kernel"


@pytest.fixture
def kernels():
    """Names of the kernels that ran since the test's start."""
    ia.ia_profile_reset()
    ia.ia_profile_enable(True)
    yield lambda: set(ia.ia_profile_report())
    ia.ia_profile_enable(False)
    ia.ia_profile_reset()


@pytest.mark.parametrize("dtype", Q.TYPES, ids=Q.ids)
@pytest.mark.parametrize("group", [64, 128])
@pytest.mark.parametrize("M,K,N", [(4000, 250, 3990), (3841, 640, 4003), (4096, 128, 3999), (3841, 100, 4003)])
def test_wide_tiles(M, K, N, group, dtype, kernels):
    """Odd sizes: rows that are no whole lines, tiles that end inside, one pair of stages and several."""
    rng = np.random.default_rng(M + K + N)
    x, w = Q._matrix(rng, M, K, dtype), q4_quantize(Q._matrix(rng, N, K, scale=K ** -0.5), group)
    bias = cuda(rng.normal(size=N).astype(np.float32))
    wide = torch.full((M, N + 20), 7.0, device="cuda", dtype=dtype)
    got = q4_linear(x, w, bias, "relu", out=wide[:, 5:5 + N])
    assert WIDE in kernels() and JOIN not in kernels()
    assert (wide[:, :5] == 7).all() and (wide[:, 5 + N:] == 7).all()
    rows = np.unique(np.concatenate([rng.integers(0, M, 60), [0, 255, 256], np.arange(M - 5, M)]))
    Q._assert_linear(got[torch.as_tensor(rows, device="cuda")], Q._f64(x)[rows], Q._values(w), Q._f64(bias), relu=True)
    assert torch.equal(got, q4_linear(x, w, bias, "relu"))


@pytest.mark.parametrize("group", [64, 128])
@pytest.mark.parametrize("M,K,N", [(1000, 4000, 4000), (2000, 8192, 2000)])
def test_wide_tiles_of_split_sums(M, K, N, group, kernels):
    rng = np.random.default_rng(M + K + N)
    x, w = Q._matrix(rng, M, K), q4_quantize(Q._matrix(rng, N, K, scale=K ** -0.5), group)
    bias = cuda(rng.normal(size=N).astype(np.float32))
    got = q4_linear(x, w, bias)
    assert {WIDE, JOIN} <= kernels()
    rows = np.unique(np.concatenate([rng.integers(0, M, 60), [0, 255, 256], np.arange(M - 5, M)]))
    Q._assert_linear(got[torch.as_tensor(rows, device="cuda")], Q._f64(x)[rows], Q._values(w), Q._f64(bias))
    assert torch.equal(got, q4_linear(x, w, bias))


@pytest.mark.parametrize("dtype", Q.TYPES, ids=Q.ids)
def test_values_that_are_not_finite(dtype, kernels):
    """NaN groups, infinite and NaN inputs stay with their output or row."""
    rng = np.random.default_rng(12)
    M, K, N = 3841, 640, 4003
    wf, x = Q._matrix(rng, N, K, scale=0.05), Q._matrix(rng, M, K, dtype)
    wf[5, 100], wf[4000, 639] = float("nan"), float("inf")
    x[17, 3], x[500, 400], x[3840, 639] = float("inf"), -float("inf"), float("nan")
    w = q4_quantize(wf, 128)
    v = Q._values(w)
    y = host(q4_linear(x, w).float())
    assert WIDE in kernels()
    assert np.isnan(y[:, [5, 4000]]).all() and np.isnan(y[3840]).all()
    rest = np.delete(np.arange(N), [5, 4000])
    for row, k, sign in ((17, 3, 1), (500, 400, -1)):
        zero = v[rest, k] == 0
        assert np.isnan(y[row, rest[zero]]).all()
        assert np.array_equal(y[row, rest[~zero]], sign * np.sign(v[rest[~zero], k]) * np.inf)
    assert np.isfinite(np.delete(y[:, rest], [17, 500, 3840], 0)).all()


SIZE = (3841, 4003)  # of the tests below, over 576 inputs


@pytest.mark.parametrize("dtype", Q.TYPES, ids=Q.ids)
def test_scales_of_any_size(dtype, kernels):
    Q.test_scales_of_any_size_and_sign(*SIZE, dtype)
    Q.test_huge_scales_over_zero_inputs(*SIZE, dtype)
    Q.test_the_largest_scales(*SIZE, dtype)
    R.test_infinite_inputs_over_scales_of_any_size(*SIZE, dtype)
    R.test_weights_of_the_whole_range(*SIZE, dtype)
    assert WIDE in kernels() and not any("few" in k or "128" in k for k in kernels())


@pytest.mark.parametrize("group", [64, 128])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=Q.ids)
def test_inputs_of_the_whole_range(dtype, group, kernels):
    R.test_inputs_near_the_largest_float(*SIZE, group, dtype)
    R.test_inputs_near_the_least_float(*SIZE, 1.0, dtype)
    assert WIDE in kernels() and not any("few" in k or "128" in k for k in kernels())


def test_fp16_scales(kernels):
    for tiny in (2.0 ** -100, -2.0 ** -66, 0.0):
        R.test_large_sums_that_cancel(*SIZE, tiny)
    for power in (-30, -24, -23, -14, 0, 8, 12):
        R.test_fp16_scales_of_every_power(*SIZE, power)
    assert WIDE in kernels() and not any("few" in k or "128" in k for k in kernels())
