"""Plain numpy definitions of table lookups and their gradient, dropout and
group-scaled 4-bit matrices, in 64 bits."""
from __future__ import annotations

import numpy as np

M32 = (1 << 32) - 1


def philox(counter, key, rounds: int = 10):
    """Philox4x32 (Salmon, Moraes, Dror & Shaw 2011) in Python's whole numbers: four words."""
    c, k = list(counter), list(key)
    for _ in range(rounds):
        a, b = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(b >> 32) ^ c[1] ^ k[0], b & M32, (a >> 32) ^ c[3] ^ k[1], a & M32]
        k = [(k[0] + 0x9E3779B9) & M32, (k[1] + 0xBB67AE85) & M32]
    return c


def words(rows: int, cols: int, seed: int, offset: int) -> np.ndarray:
    """[rows, cols] words: the one that decides on each value of a matrix (in uint64)."""
    quads = (cols + 3) // 4
    c = [np.tile(np.arange(quads, dtype=np.uint64), rows), np.repeat(np.arange(rows, dtype=np.uint64), quads),
         np.full(rows * quads, offset & M32, np.uint64), np.full(rows * quads, offset >> 32, np.uint64)]
    k = [seed & M32, seed >> 32]
    low, high = np.uint64(M32), np.uint64(32)
    for _ in range(10):
        a, b = np.uint64(0xD2511F53) * c[0], np.uint64(0xCD9E8D57) * c[2]
        c = [(b >> high) ^ c[1] ^ np.uint64(k[0]), b & low, (a >> high) ^ c[3] ^ np.uint64(k[1]), a & low]
        k = [(k[0] + 0x9E3779B9) & M32, (k[1] + 0xBB67AE85) & M32]
    return np.stack(c, 1).reshape(rows, 4 * quads)[:, :cols]


def kept(rows: int, cols: int, p: float, seed: int, offset: int = 0) -> np.ndarray:
    return words(rows, cols, seed, offset) >= np.uint64(round(p * 2.0 ** 32))


def dropout(x, p, seed, offset=0):
    x = np.asarray(x, np.float64)
    on = kept(*x.shape, p, seed, offset)
    return np.where(on, x / (1.0 - p) if p < 1.0 else 0.0, 0.0)


def lookup(table, index, scale=1.0, p=0.0, seed=0, offset=0):
    table, index = np.asarray(table, np.float64), np.asarray(index, np.int64)
    out = np.zeros((len(index), table.shape[1]))
    for i, v in enumerate(index):
        if 0 <= v < len(table):
            out[i] = scale * table[v]
    return dropout(out, p, seed, offset) if p else out


def lookup_gradient(dy, index, entries, scale=1.0, p=0.0, seed=0, offset=0):
    """(gradient, sums of magnitudes, rows of each entry)."""
    d, index = np.asarray(dy, np.float64) * scale, np.asarray(index, np.int64)
    if p:
        d = dropout(d, p, seed, offset)
    g, size, count = np.zeros((entries, d.shape[1])), np.zeros((entries, d.shape[1])), np.zeros(entries, np.int64)
    on = (index >= 0) & (index < entries)
    np.add.at(g, index[on], d[on])
    np.add.at(size, index[on], np.abs(d[on]))
    np.add.at(count, index[on], 1)
    return g, size, count


def q4_quantize(x, group: int):
    """(q [rows, groups, group], z, s [rows, groups]) of a matrix, in 64 bits."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    groups = -(-cols // group)
    q, z, s = np.zeros((rows, groups, group)), np.zeros((rows, groups)), np.zeros((rows, groups))
    for r in range(rows):
        for g in range(groups):
            v = np.zeros(group)
            part = x[r, g * group:(g + 1) * group]
            v[:len(part)] = part
            if not np.isfinite(v).all():
                s[r, g] = np.nan
                continue
            lo, hi = min(0.0, v.min()), max(0.0, v.max())
            if lo == hi:
                continue
            m, e = np.frexp((hi - lo) / 15.0)
            unit = max(np.ldexp(np.ceil(m * 65536.0), e - 16), 2.0 ** -100)
            zero = np.rint(-lo / unit)
            q[r, g], z[r, g], s[r, g] = np.clip(np.rint(v / unit) + zero, 0, 15), zero, unit
    return q, z, s


def q4_pack(q, z, s):
    """(codes, words) of the format."""
    rows, groups, group = q.shape
    c = q.astype(np.uint8).reshape(rows, groups * group)
    bits = np.where(np.isnan(s), np.float32(np.nan), s).astype(np.float32).view(np.uint32)
    bits = np.where(np.isnan(s), np.uint32(0x7FC00000), bits)
    assert not (bits & 255).any()
    w = np.zeros((rows, -(-groups // 4) * 4), np.uint32)
    w[:, :groups] = bits | z.astype(np.uint32)
    return c[:, 0::2] | (c[:, 1::2] << 4), w.view(np.int32)


def q4_values(codes, words_, cols: int, group: int):
    """The values that packed rows stand for."""
    rows = len(codes)
    q = np.stack([codes & 15, codes >> 4], -1).reshape(rows, -1, group).astype(np.float64)
    w = words_.view(np.uint32)[:, :q.shape[1], None]
    s = (w & np.uint32(0xFFFFFF00)).view(np.float32).astype(np.float64)
    return (s * (q - (w & np.uint32(255)))).reshape(rows, -1)[:, :cols]
