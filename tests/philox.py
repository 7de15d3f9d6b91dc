"""Philox-4x32 with ten rounds (Salmon, Moraes, Dror, Shaw 2011), in plain numpy, and
the dropout mask that is made of it."""
import numpy as np

LOW = np.uint64(0xFFFFFFFF)


def philox(counter, key):
    """uint32 [n, 4] for a counter of four words (arrays or numbers) and a key of two."""
    c = [np.asarray(x, np.uint64) for x in counter]
    k = [int(x) for x in key]
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [b >> np.uint64(32) ^ c[1] ^ np.uint64(k[0]), b & LOW,
             a >> np.uint64(32) ^ c[3] ^ np.uint64(k[1]), a & LOW]
        k = [k[0] + 0x9E3779B9 & 0xFFFFFFFF, k[1] + 0xBB67AE85 & 0xFFFFFFFF]
    return np.stack(np.broadcast_arrays(*c), -1).astype(np.uint32)


def parts(t, D, seed, offset):
    """The 16-bit parts [len(t), D] of tokens t (an array of indices)."""
    groups = (D + 7) // 8
    at = (np.asarray(t, np.uint64)[:, None] * np.uint64(groups) + np.arange(groups, dtype=np.uint64)).reshape(-1)
    seed, offset = seed % (1 << 64), offset % (1 << 64)
    w = philox((at & LOW, at >> np.uint64(32), offset & 0xFFFFFFFF, offset >> 32),
               (seed & 0xFFFFFFFF, seed >> 32))
    return np.stack([w & 0xFFFF, w >> 16], -1).reshape(len(t), groups * 8)[:, :D]


def kept(t, D, p, seed, offset):
    """(what is kept [len(t), D], the factor of what is kept)."""
    n = int(np.floor(65536 * p + 0.5))
    return parts(t, D, seed, offset) >= n, 65536 / (65536 - n) if n < 65536 else 0.0
