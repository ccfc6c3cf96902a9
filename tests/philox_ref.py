"""Dropout from the definition, in numpy: Philox 4x32-10 in 64-bit integers."""
import numpy as np


def philox(counter, key, rounds=10):
    """The 4 words (uint64 arrays below 2^32) of blocks whose 4 counter words are given."""
    c = [np.asarray(v, dtype=np.uint64) for v in counter]
    k = [int(v) for v in key]
    low = np.uint64(0xFFFFFFFF)
    sh = np.uint64(32)
    for _ in range(rounds):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> sh) ^ c[1] ^ np.uint64(k[0]), b & low, (a >> sh) ^ c[3] ^ np.uint64(k[1]), a & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def words(n, seed, offset=0, first=0):
    """Words first .. first + n - 1 of the tensor's stream (first a multiple of 4)."""
    g = np.arange(first // 4, (first + n + 3) // 4, dtype=np.uint64)
    one = np.ones_like(g)
    c = philox((g & np.uint64(0xFFFFFFFF), g >> np.uint64(32), one * np.uint64(offset & 0xFFFFFFFF),
                one * np.uint64((offset >> 32) & 0xFFFFFFFF)),
               (seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF))
    return np.stack(c, 1).reshape(-1)[:n]


def keep(n, p, seed, offset=0, first=0):
    if p == 1.0:
        return np.zeros(n, dtype=bool)
    return words(n, seed, offset, first) >= np.uint64(int(p * 2.0 ** 32))
