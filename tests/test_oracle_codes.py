"""The oracle of lookups, dropout and group-scaled 4 bits: the generator's
published answers, closed forms and differences."""
import numpy as np
import pytest

from oracle import codes as O


@pytest.mark.parametrize("counter,key,want", [
    ([0] * 4, [0] * 2, [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]),
    ([0xFFFFFFFF] * 4, [0xFFFFFFFF] * 2, [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]),
    ([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0],
     [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]),
])
def test_philox_gives_the_published_answers(counter, key, want):
    """The known answers that the generator's authors publish for ten rounds."""
    assert O.philox(counter, key) == want


def test_words_are_the_generators_at_their_place():
    seed, offset = 0x123456789ABCDEF0, 0xFEDCBA9876543210
    w = O.words(5, 11, seed, offset)
    for r in (0, 1, 4):
        for c in (0, 3, 4, 10):
            want = O.philox([c // 4, r, offset & O.M32, offset >> 32], [seed & O.M32, seed >> 32])[c % 4]
            assert int(w[r, c]) == want


def test_dropout_keeps_its_share():
    x = np.ones((400, 500))
    for p in (0.1, 0.5, 0.9):
        y = O.dropout(x, p, 3, 1)
        share = (y != 0).mean()
        assert abs(share - (1 - p)) < 5 * np.sqrt(p * (1 - p) / x.size)  # five standard deviations
        assert np.allclose(y[y != 0], 1 / (1 - p))
    assert (O.dropout(x, 0.0, 3) == 1).all() and (O.dropout(x, 1.0, 3) == 0).all()
    assert (O.kept(50, 50, 0.5, 3, 1) != O.kept(50, 50, 0.5, 3, 2)).any()


def test_lookup_gradient_by_differences():
    """The lookup is linear in the table: a unit step of one value moves sum(dy * out) by its gradient."""
    rng = np.random.default_rng(0)
    table, dy = rng.normal(size=(6, 5)), rng.normal(size=(9, 5))
    index = np.array([0, 5, 5, -1, 2, 6, 5, 0, 3])
    g, size, count = O.lookup_gradient(dy, index, 6, 1.5, 0.3, 7, 2)
    base = (dy * O.lookup(table, index, 1.5, 0.3, 7, 2)).sum()
    for v in range(6):
        for c in range(5):
            t = table.copy()
            t[v, c] += 1.0
            assert abs((dy * O.lookup(t, index, 1.5, 0.3, 7, 2)).sum() - base - g[v, c]) < 1e-12
    assert count.tolist() == [2, 0, 1, 1, 0, 3] and (np.abs(g) <= size + 1e-15).all()


@pytest.mark.parametrize("group", [32, 64, 128])
def test_quantised_values_are_near(group):
    rng = np.random.default_rng(group)
    x = rng.normal(size=(7, 300)) * np.exp(rng.normal(size=(7, 1)))
    q, z, s = O.q4_quantize(x, group)
    codes, words = O.q4_pack(q, z, s)
    v = O.q4_values(codes, words, 300, group)
    unit = np.repeat(s, group, 1)[:, :300]
    # half a step, also where a code is held to 15: hi / s <= 15 + lo / s and z <= -lo / s + 1/2, so s (15 - z) >= hi - s / 2
    assert (np.abs(v - x) <= 0.5 * unit * (1 + 1e-12)).all()
    assert q.min() >= 0 and q.max() <= 15 and z.min() >= 0 and z.max() <= 15


def test_quantised_whole_steps_are_exact():
    """Values that are whole multiples of a 16-bit scale come back as they are."""
    x = (np.arange(32) % 16 - 5.0)[None] * 0.375
    assert (O.q4_values(*O.q4_pack(*O.q4_quantize(x, 32)), 32, 32) == x).all()
    bad = x.copy()
    bad[0, 3] = np.inf
    assert np.isnan(O.q4_values(*O.q4_pack(*O.q4_quantize(bad, 32)), 32, 32)).all()
    assert (O.q4_values(*O.q4_pack(*O.q4_quantize(0 * x, 32)), 32, 32) == 0).all()
