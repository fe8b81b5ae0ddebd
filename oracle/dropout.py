"""fp64 dropout from a counter-based generator (test infrastructure only).

The generator is Philox-4x32 with 10 rounds, written from the paper (Salmon,
Moraes, Dror, Shaw: "Parallel random numbers: as easy as 1, 2, 3", 2011) in
plain Python integers for one counter and in numpy uint64 for arrays.

Mask layout: eight columns of a row share one counter
(b, b >> 32, offset, offset >> 32 in 32-bit words) with
b = row * ceil(cols / 8) + col // 8; the low and high 16 bits of word j
belong to columns 2j and 2j + 1 of the eight.  An element is kept where its
16 bits are at least t = round(65536 p).
"""

import numpy as np

M0, M1 = 0xD2511F53, 0xCD9E8D57
W0, W1 = 0x9E3779B9, 0xBB67AE85
LOW = 0xFFFFFFFF


def philox4x32(counter, key, rounds=10):
    """The four output words of one counter (Python integers)."""
    c, k = list(counter), list(key)
    for _ in range(rounds):
        a, b = M0 * c[0], M1 * c[2]
        c = [(b >> 32) ^ c[1] ^ k[0], b & LOW, (a >> 32) ^ c[3] ^ k[1], a & LOW]
        k = [(k[0] + W0) & LOW, (k[1] + W1) & LOW]
    return c


def threshold(p):
    return int(np.floor(65536.0 * p + 0.5))


def factor(p):
    t = threshold(p)
    return 0.0 if t >= 65536 else 65536.0 / (65536 - t)


def mask(rows, cols, p, seed, offset):
    """Boolean [rows, cols]: True where the element is kept."""
    nv = -(-cols // 8)
    b = np.arange(rows * nv, dtype=np.uint64)
    low, sh = np.uint64(LOW), np.uint64(32)
    c = [b & low, b >> sh, np.full_like(b, offset & LOW), np.full_like(b, (offset >> 32) & LOW)]
    k = [seed & LOW, (seed >> 32) & LOW]
    for _ in range(10):
        m0, m1 = c[0] * np.uint64(M0), c[2] * np.uint64(M1)
        c = [(m1 >> sh) ^ c[1] ^ np.uint64(k[0]), m1 & low, (m0 >> sh) ^ c[3] ^ np.uint64(k[1]), m0 & low]
        k = [(k[0] + W0) & LOW, (k[1] + W1) & LOW]
    bits = np.empty((rows * nv, 8), dtype=np.int64)
    for j in range(4):
        bits[:, 2 * j] = c[j] & np.uint64(0xFFFF)
        bits[:, 2 * j + 1] = c[j] >> np.uint64(16)
    return (bits >= threshold(p)).reshape(rows, nv * 8)[:, :cols]


def dropout(x, p, seed, offset, residual=None):
    """(y, |terms|): residual + mask * x * factor in fp64."""
    x = np.asarray(x, dtype=np.float64)
    y = np.where(mask(*x.shape, p, seed, offset), x * factor(p), 0.0) if threshold(p) else x.copy()
    mag = np.abs(y)
    if residual is not None:
        r = np.asarray(residual, dtype=np.float64)
        y, mag = y + r, mag + np.abs(r)
    return y, mag
