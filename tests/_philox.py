"""Philox 4x32-10 (Salmon et al. 2011) in NumPy's 64-bit arithmetic, and the
dropout mask that the library defines with it."""

import numpy as np


def philox(counter, key):
    """Four uint64 arrays of 32-bit words for four of the counter and two of the key."""
    m32 = np.uint64(0xFFFFFFFF)
    c = [np.asarray(v, dtype=np.uint64) for v in counter]
    k = [int(v) for v in key]
    for _ in range(10):
        a, b = np.uint64(0xD2511F53) * c[0], np.uint64(0xCD9E8D57) * c[2]
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), b & m32, (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), a & m32]
        k = [(k[0] + 0x9E3779B9) % 2 ** 32, (k[1] + 0xBB67AE85) % 2 ** 32]
    return c


def kept(n, dim, p, seed, offset, rows=False):
    seed, offset = seed % 2 ** 64, offset % 2 ** 64
    columns = 1 if rows else dim
    row, col = np.meshgrid(np.arange(n), np.arange((columns + 3) // 4), indexing="ij")
    w = philox([col, row, np.full(row.shape, offset % 2 ** 32), np.full(row.shape, offset >> 32)],
               (seed % 2 ** 32, seed >> 32))
    words = np.stack(w, 2).reshape(n, 4 * ((columns + 3) // 4))[:, :columns]
    return np.broadcast_to(words >= np.uint64(round(p * 2 ** 32)), (n, dim))
