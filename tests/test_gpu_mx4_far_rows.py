"""Gradients of narrow layers whose rows lie 2^22 elements and more apart,
against the same rows beside each other: bit for bit."""
import numpy as np
import pytest
import torch

from implicit_attribute_decode_amd.pipeline import mx4_linear_backward, mx4_quantize

pytestmark = pytest.mark.gpu

FAR = (1 << 22) + 8


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16], ids=lambda v: str(v)[6:])
@pytest.mark.parametrize("M,N,K", [(1, 4, 4), (31, 58, 70), (128, 256, 192), (300, 250, 33), (515, 5, 256)])
def test_far_rows_equal_near_ones(M, N, K, dtype):
    gen = torch.Generator(device="cuda").manual_seed(M)
    new = lambda *s: torch.randn(s, generator=gen, device="cuda").to(dtype)  # noqa: E731
    dy, x, y = new(M, N), new(M, K), new(M, N).relu()
    wt = mx4_quantize(new(N, K), transpose=True)
    room = torch.full((3 * 512 + M * FAR,), float("nan"), dtype=dtype, device="cuda")
    apart = lambda t, k: room.as_strided(tuple(t.shape), (FAR, 1), 513 * k).copy_(t)  # noqa: E731
    dyf, xf, yf = apart(dy, 0), apart(x, 1), apart(y, 2)
    for mask, maskf in ((None, None), (y, yf)):
        want = mx4_linear_backward(dy, x, wt, mask)
        for a, b in ((dyf, x), (dy, xf), (dyf, xf)):
            got = mx4_linear_backward(a, b, wt, maskf)
            assert all(torch.equal(got[k], want[k]) for k in want)
        part = mx4_linear_backward(dyf, x, None, maskf, want_x=False)
        assert torch.equal(part["weight"], want["weight"]) and torch.equal(part["bias"], want["bias"])
