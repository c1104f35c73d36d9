"""MXFP4 layers and gradients of so many rows that the kernels' loops over rows
repeat: the narrow gradient's blocks take several steps of 128 rows (from 32,769
rows on) with a ragged last one, the narrow layer's blocks several rounds (from
65,537 rows on at 256 x 256, 131,073 in small layers).

Operands are E2M1 values, which every block holds exactly, of either sign, and
biases whole numbers: every partial sum is a multiple of 1/4 far below 2^22, so
exact in fp32.  Gradients of weights and biases therefore equal the sums in 64
bits, outputs their one rounding."""
import pytest
import torch

from implicit_attribute_decode_amd import ia
from implicit_attribute_decode_amd.pipeline import mx4_linear, mx4_linear_backward, mx4_quantize

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.float16, torch.bfloat16]
ids = lambda v: str(v).replace("torch.", "") if isinstance(v, torch.dtype) else None  # noqa: E731


def _grid(gen, *shape):
    """E2M1 values of either sign, zeros among them."""
    values = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0], device="cuda")
    return values[torch.randint(0, 15, shape, generator=gen, device="cuda")]


def _product(a, b):
    """a b^T in 64 bits, a's rows a part at a time."""
    bt = b.double().t().contiguous()
    return torch.cat([part.double() @ bt for part in a.split(1 << 17)])


def _columns(d, x):
    """d^T x in 64 bits."""
    out = torch.zeros((d.shape[1], x.shape[1]), dtype=torch.float64, device="cuda")
    for a, b in zip(d.split(1 << 17), x.split(1 << 17)):
        out += a.double().t().contiguous() @ b.double()
    return out


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("relu", [False, True])
@pytest.mark.parametrize("M,N,K", [(32_769, 256, 192), (70_001, 58, 250), (300_007, 256, 192), (300_007, 58, 250),
                                   (1_200_033, 12, 33), (33_000, 4, 256), (98_305, 255, 5)])
def test_narrow_gradients_of_many_rows(M, N, K, relu, dtype):
    gen = torch.Generator(device="cuda").manual_seed(M + N + relu)
    x, dy, w = _grid(gen, M, K).to(dtype), _grid(gen, M, N).to(dtype), _grid(gen, N, K)
    y = _grid(gen, M, N).relu().to(dtype) if relu else None
    got = mx4_linear_backward(dy, x, mx4_quantize(w, transpose=True), y)
    d = torch.where(y > 0, dy, torch.zeros_like(dy)) if relu else dy
    assert torch.equal(got["x"], _product(d, w.t()).to(dtype))
    assert torch.equal(got["weight"].double(), _columns(d, x))
    assert torch.equal(got["bias"].double(), _columns(d, torch.ones_like(x[:, :1])).view(-1))
    part = mx4_linear_backward(dy, x, None, y, want_x=False)
    assert torch.equal(part["weight"], got["weight"]) and torch.equal(part["bias"], got["bias"])


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("M,N,K", [(20_003, 600, 64), (16_384, 300, 250), (16_383, 300, 250), (40_001, 1700, 11)])
def test_gradients_of_wide_upstream_rows(M, N, K, dtype):
    """More than 256 outputs back to few inputs."""
    gen = torch.Generator(device="cuda").manual_seed(M)
    x, dy, w, y = _grid(gen, M, K).to(dtype), _grid(gen, M, N).to(dtype), _grid(gen, N, K), _grid(gen, M, N).relu().to(dtype)
    got = mx4_linear_backward(dy, x, mx4_quantize(w, transpose=True), y)
    d = torch.where(y > 0, dy, torch.zeros_like(dy))
    assert torch.equal(got["x"], _product(d, w.t()).to(dtype))
    assert torch.equal(got["weight"].double(), _columns(d, x))
    assert torch.equal(got["bias"].double(), _columns(d, torch.ones_like(x[:, :1])).view(-1))


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("M,N,K", [(131_073, 64, 64), (300_007, 64, 32), (600_011, 11, 100), (65_537, 256, 256),
                                   (200_003, 250, 131), (140_001, 1000, 200)])
def test_narrow_layers_of_many_rows(M, N, K, dtype):
    gen = torch.Generator(device="cuda").manual_seed(N + K)
    x, w = _grid(gen, M, K).to(dtype), _grid(gen, N, K)
    bias = torch.randint(-50, 50, (N,), generator=gen, device="cuda").float()
    want = (_product(x, w) + bias.double()).relu()
    out = torch.full((M, N + 3), 7.0, device="cuda", dtype=dtype)
    for to in (None, out[:, 1:1 + N]):
        assert torch.equal(mx4_linear(x, mx4_quantize(w), bias, "relu", out=to), want.to(dtype))
    assert (out[:, 0] == 7).all() and (out[:, 1 + N:] == 7).all()


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("M,N,K", [(5000, 64, 300), (5000, 65, 300), (3001, 40, 2000), (20_001, 250, 2), (700, 817, 18)])
def test_gradients_of_one_wide_side(M, N, K, dtype):
    """The input's gradient alone and beside the others: the same bits whichever way d is quantised."""
    gen = torch.Generator(device="cuda").manual_seed(N)
    x, dy, w, y = _grid(gen, M, K).to(dtype), _grid(gen, M, N).to(dtype), _grid(gen, N, K), _grid(gen, M, N).relu().to(dtype)
    wt = mx4_quantize(w, transpose=True)
    got = mx4_linear_backward(dy, x, wt, y)
    d = torch.where(y > 0, dy, torch.zeros_like(dy))
    assert torch.equal(got["x"], _product(d, w.t()).to(dtype))
    assert torch.equal(got["weight"].double(), _columns(d, x))
    assert torch.equal(got["bias"].double(), _columns(d, torch.ones_like(x[:, :1])).view(-1))
    n = ia.ia_mx4_linear_backward_workspace_size(M, N, K)
    dx = torch.full((M, K), 7.0, dtype=dtype, device="cuda")
    ia.ia_mx4_linear_backward(dy, N, y, N, None, 0, {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}[dtype], M, N, K,
                              wt.c, dx, K, None, None, torch.empty(n, dtype=torch.uint8, device="cuda"))
    assert torch.equal(dx, got["x"])
