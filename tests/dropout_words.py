"""The dropout calls' random words on the CPU: Philox4x32 of 10 rounds in numpy (Salmon, Moraes,
Dror, Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011)."""
import math

import numpy as np

LOW = np.uint64(0xFFFFFFFF)


def philox(counter, key):
    """Four arrays of 32-bit counter words and two key words to four arrays of output words."""
    c = [np.asarray(x, dtype=np.uint64) for x in counter]
    k = [int(x) for x in key]
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), b & LOW,
             (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), a & LOW]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def words(elements, seed, draw):
    """The 16-bit word of each element index."""
    i = np.asarray(elements, dtype=np.uint64)
    q, lane = i >> np.uint64(3), (i & np.uint64(7)).astype(np.int64)
    out = np.stack(philox([q & LOW, q >> np.uint64(32), np.full_like(q, draw & 0xFFFFFFFF),
                           np.full_like(q, draw >> 32)], [seed & 0xFFFFFFFF, seed >> 32]))
    word = np.take_along_axis(out, lane[None] >> 1, 0)[0]
    return (word >> (np.uint64(16) * (lane & 1).astype(np.uint64))) & np.uint64(0xFFFF)


def threshold(rate):
    return math.floor(rate * 65536 + 0.5)


def dropped(x, rate, seed, draw, first=0):
    """Dropout of x (any shape) in 64 bits; `first`: the index of its first element."""
    x = np.asarray(x, dtype=np.float64)
    t = threshold(rate)
    keep = (words(np.arange(first, first + x.size), seed, draw) >= t).reshape(x.shape)
    return np.where(keep, x * (65536.0 / (65536 - t) if t < 65536 else 0.0), 0.0), keep
