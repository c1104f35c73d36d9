"""Lookups, table gradients, dropout and 4-bit conversions at the sizes where they take another way: four rows a
thread, stores past the memory-side cache, longer tiles of sorted rows, more than one tile of the sort in a block,
eight columns a lane, second launches.  References in 64 bits; tolerances:
test_gpu_embedding.py's and test_gpu_dropout.py's."""
import functools

import numpy as np
import pytest
import torch

from oracle import codes as O
from implicit_attribute_decode_amd.pipeline import Dropout, embedding, embedding_backward, mx4_quantize, q4_quantize

from test_gpu_embedding import TINY, TYPES, UNIT, ids

pytestmark = pytest.mark.gpu


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(seed, *shape, dtype=torch.float32):
    return torch.randn(shape, generator=_gen(seed), device="cuda").to(dtype)


@functools.lru_cache(maxsize=4)
def _oracle(rows, cols, p, seed, offset):
    return torch.as_tensor(O.kept(rows, cols, p, seed, offset))


def _kept(rows, cols, d):
    return _oracle(rows, cols, d.p, d.seed, d.offset).cuda()


def _assert_values(got, want):
    """One fp32 product by an fp32 factor, then half a step of the type."""
    tol = (2 * 2.0 ** -24 + UNIT[got.dtype]) * (1 + 2.0 ** -10) * want.abs() + TINY[got.dtype]
    assert bool(((got.double() - want).abs() <= tol).all())


# Eight values a thread: four rows each from 2^21 threads on; outputs of 64 MB pass by the memory-side cache
LARGE = [(300_001, 57), (300_001, 120), (2_100_000, 5)]


@pytest.mark.parametrize("table", ["f32", "f16", "bf16", "mx4"])
@pytest.mark.parametrize("n,dim", LARGE)
def test_large_lookups(n, dim, table):
    values = _randn(1, 5000, dim)
    if table == "mx4":
        t = mx4_quantize(values)
        values = t.dequantize()
    else:
        t = values = values.to({"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[table])
    index = torch.randint(-50, 5060, (n,), generator=_gen(2), device="cuda")
    index[-1], index[0] = 4999, -1
    there = ((index >= 0) & (index < 5000)).unsqueeze(1)
    rows = torch.where(there, values[index.clamp(0, 4999)].double(), 0.0)
    wide = torch.full((n, dim + 9), 7.0, device="cuda", dtype=torch.float16)
    embedding(t, index, 1.25, out=wide[:, 3:3 + dim])
    _assert_values(wide[:, 3:3 + dim], rows * 1.25)
    assert bool((wide[:, :3] == 7).all()) and bool((wide[:, 3 + dim:] == 7).all())
    d = Dropout(0.3, 2 ** 63 + 5, 2 ** 35 + 1)
    got = embedding(t, index.to(torch.int32), 0.5, torch.float32, d)
    _assert_values(got, torch.where(_kept(n, dim, d), rows * (0.5 / 0.7), 0.0))


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
def test_large_dropout_into_a_wider_array(dtype):
    rows, cols = 300_001, 250
    x = _randn(3, rows, cols, dtype=dtype)
    d = Dropout(0.4, 11, 3)
    wide = torch.full((rows, 259), 7.0, device="cuda", dtype=dtype)
    d(x, out=wide[:, 3:253])
    _assert_values(wide[:, 3:253], torch.where(_kept(rows, cols, d), x.double() / 0.6, 0.0))
    assert bool((wide[:, :3] == 7).all()) and bool((wide[:, 253:] == 7).all())


# ------------------------------------------------------------------ gradient


def _assert_gradient(dy, index, entries, scale=1.0, d=None):
    """Against sums in 64 bits on the CPU: at most 64 fp32 sums in a row, and a product."""
    rows = dy.double().cpu() * scale
    if d is not None:
        rows = torch.where(_oracle(*dy.shape, d.p, d.seed, d.offset), rows / (1.0 - d.p), 0.0)
    at = index.long().cpu()
    on = (at >= 0) & (at < entries)
    want = torch.zeros((entries, dy.shape[1]), dtype=torch.float64)
    size = want.clone()
    want.index_add_(0, at[on], rows[on])
    size.index_add_(0, at[on], rows[on].abs())
    got = embedding_backward(dy, index, entries, scale, d)
    assert got.dtype == torch.float32
    assert bool(((got.double().cpu() - want).abs() <= 67 * 2.0 ** -24 * size + 2.0 ** -149).all())
    assert torch.equal(got, embedding_backward(dy, index, entries, scale, d))


def _index(kind, n, entries):
    if kind == "one":
        return torch.full((n,), entries - 1, device="cuda")
    if kind == "none":
        return torch.full((n,), -1, device="cuda")
    i = torch.randint(-1, entries + 1, (n,), generator=_gen(4), device="cuda")
    if kind == "sorted":
        i = i.sort().values
    if kind == "few":
        i = torch.where(torch.rand(n, generator=_gen(5), device="cuda") < 0.7, i % 3, i)
    return i


@pytest.mark.parametrize("kind", ["random", "sorted", "one", "few", "none"])
@pytest.mark.parametrize("dtype", TYPES, ids=ids)
def test_longer_tiles_of_sorted_rows(kind, dtype):
    """270,000 rows of 250 values: tiles of 32 rows."""
    dy = _randn(6, 270_000, 250, dtype=dtype)
    _assert_gradient(dy, _index(kind, 270_000, 9000), 9000, 1.5)
    _assert_gradient(dy, _index(kind, 270_000, 150).to(torch.int32), 150, 1.0, Dropout(0.2, 9, 2))


@pytest.mark.parametrize("kind", ["random", "sorted", "one", "few"])
@pytest.mark.parametrize("n,dim,entries", [(600_000, 4, 70_000), (1_300_000, 1, 300), (530_000, 7, 5_000_000)])
def test_blocks_that_sort_several_tiles(kind, n, dim, entries):
    dy = _randn(7, n, dim)
    _assert_gradient(dy, _index(kind, n, entries), entries)


@pytest.mark.parametrize("kind", ["random", "one", "few"])
@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("dim", [257, 512, 513, 514, 515, 1030])
def test_wide_rows(dim, dtype, kind):
    """Eight columns a lane, rows of any number of values."""
    wide = _randn(8, 5000, dim + 3, dtype=dtype)
    dy = wide[:, 1:1 + dim]
    _assert_gradient(dy, _index(kind, 5000, 300), 300, 0.5)
    _assert_gradient(dy, _index(kind, 5000, 300), 300, 0.5, Dropout(0.6, 2 ** 50, 7))


# ---------------------------------------------------------- second launches


def _last_words(rows, first, d):
    """The words that decide on column 0 of rows first.., of a matrix of `rows`."""
    return np.array([O.philox([0, r, d.offset & O.M32, d.offset >> 32], [d.seed & O.M32, d.seed >> 32])[0]
                     for r in range(first, rows)])


def test_the_most_rows():
    """2^31 - 1 rows of one value: a launch takes 2^31 - 256 threads, the last 255 rows go in another."""
    n, tail = 2 ** 31 - 1, 600
    d = Dropout(0.5, 77, 2 ** 33 + 9)
    kept = torch.as_tensor(_last_words(n, n - tail, d) >= 2 ** 31, device="cuda")
    x = torch.tensor([[3.0]], dtype=torch.bfloat16, device="cuda").expand(n, 1)
    y = d(x)
    assert torch.equal(y[-tail:, 0], torch.where(kept, 6.0, 0.0).to(torch.bfloat16))
    y.fill_(7)
    table = torch.tensor([[1.0], [5.0]], dtype=torch.bfloat16, device="cuda")
    index = torch.tensor([1], device="cuda").expand(n)
    embedding(table, index, out=y)
    assert bool((y[-tail:] == 5).all()) and bool((y[:tail] == 5).all())
    embedding(table, index, dropout=d, out=y)
    assert torch.equal(y[-tail:, 0], torch.where(kept, 10.0, 0.0).to(torch.bfloat16))
    # about half of all: six standard deviations of a share of 2^31
    share = sum(int((part != 0).sum()) for part in y.split(2 ** 28)) / n
    assert abs(share - 0.5) < 6 * 0.5 / n ** 0.5


def test_gradient_of_the_most_rows():
    """2^31 - 1 rows of 129 values (one row repeated) of one entry: 2^24 blocks of tiles, 2^32 threads (105 GB of workspace)."""
    n = 2 ** 31 - 1
    dy = (torch.arange(129, device="cuda") % 3 - 1).to(torch.bfloat16).view(1, 129).expand(n, 129)
    g = embedding_backward(dy, torch.tensor([1], dtype=torch.int32, device="cuda").expand(n), 3)
    # sums of whole numbers: exact in a tile and in the join in double, then 2^31 - 1 rounds to 2^31
    assert torch.equal(g[1], dy[0].float() * 2.0 ** 31) and not bool(g[0].any()) and not bool(g[2].any())


def test_4_bit_conversions_in_several_launches():
    """2^29 + 100 rows of one value in groups of 32: a launch takes 2^29 - 64 of them."""
    n = 2 ** 29 + 100
    one = torch.tensor([[-3.0]], dtype=torch.bfloat16, device="cuda")
    q, want = q4_quantize(one.expand(n, 1), 32), q4_quantize(one, 32)
    for rows in (slice(0, 300), slice(n - 300, n)):
        assert torch.equal(q.codes[rows], want.codes.expand(300, -1)) and torch.equal(q.words[rows], want.words.expand(300, -1))
    y, value = q.dequantize(torch.bfloat16), want.dequantize(torch.bfloat16)
    assert bool((y[:300] == value).all()) and bool((y[-300:] == value).all())


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
def test_large_read_back_into_a_wider_array(dtype):
    """Outputs past the memory-side cache at any place; words and codes against the definition in 64 bits."""
    rows, cols, group = 5003, 7001, 64
    x = _randn(10, rows, cols, dtype=dtype)
    q = q4_quantize(x, group)
    groups = -(-cols // group)
    v = np.zeros((rows, groups * group))
    v[:, :cols] = x.double().cpu().numpy()
    v = v.reshape(rows, groups, group)
    lo, hi = np.minimum(v.min(-1), 0), np.maximum(v.max(-1), 0)
    m, e = np.frexp((hi - lo) / 15.0)
    s = np.ldexp(np.ceil(m * 65536.0), e - 16)  # no group of these is of zeros
    z = np.rint(-lo / s)
    codes, words = O.q4_pack(np.clip(np.rint(v / s[..., None]) + z[..., None], 0, 15), z, s)
    assert np.array_equal(q.codes.cpu().numpy(), codes) and np.array_equal(q.words.cpu().numpy(), words)
    wide = torch.full((rows, cols + 10), 7.0, device="cuda", dtype=dtype)
    q.dequantize(out=wide[:, 3:3 + cols])
    want = torch.as_tensor(O.q4_values(codes, words, cols, group)).to(dtype)
    assert torch.equal(wide[:, 3:3 + cols].cpu(), want)
    assert bool((wide[:, :3] == 7).all()) and bool((wide[:, 3 + cols:] == 7).all())
