"""The bias gradient over very many rows.

A block of 32 rows is summed in fp32 (31 additions, eight such sums joined in the
wide layers: 7 more), everything above that in double and rounded twice to fp32:
40 roundings of at most 2^-24 of the sum of magnitudes, however many rows there
are; 42 with the last one and a margin."""
import numpy as np
import pytest
import torch

from implicit_attribute_decode_amd.pipeline import mx4_linear_backward

from gpu_util import say

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.float16, torch.bfloat16]
ids = lambda v: str(v).replace("torch.", "") if isinstance(v, torch.dtype) else None  # noqa: E731


def _check(dy, x, y=None):
    db = mx4_linear_backward(dy, x, None, y, want_x=False)["bias"].double()
    d = dy if y is None else torch.where(y > 0, dy, torch.zeros_like(dy))
    want, scale = torch.zeros_like(db), torch.zeros_like(db)
    for part in d.split(1 << 20):
        want += part.double().sum(0)
        scale += part.double().abs().sum(0)
    worst = float(((db - want).abs() / scale).max() * 2.0 ** 24)
    say(f"{tuple(dy.shape)} {dy.dtype}: {worst:.2f} x 2^-24 of the magnitudes")
    assert worst <= 42.0


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("M,N,K", [(8_000_003, 8, 4), (3_000_017, 5, 70), (1_000_003, 300, 8)])
def test_one_row_repeated(M, N, K, dtype):
    """A sum's gradient: every row alike, so that rounding errors have one sign."""
    row = torch.linspace(0.1, 0.9, N, device="cuda").to(dtype)
    _check(row.expand(M, N), torch.ones(K, device="cuda", dtype=dtype).expand(M, K))


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("M,N,K", [(2_000_003, 58, 8), (700_001, 250, 4)])
def test_random_gradients_under_a_mask(M, N, K, dtype):
    gen = torch.Generator(device="cuda").manual_seed(4)
    dy = torch.rand((M, N), generator=gen, device="cuda").add_(0.5).to(dtype)
    y = torch.randn((M, N), generator=gen, device="cuda").relu_().to(dtype)
    _check(dy, torch.ones(K, device="cuda", dtype=dtype).expand(M, K), y)
