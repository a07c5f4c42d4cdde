"""Counter-based dropout, written plainly on the CPU (numpy): the mask as the
definition in include/drop.h reads, one element at a time in whole arrays, and
the products in Python's or numpy's 64-bit integers.  Shares no code with the
HIP path."""
from __future__ import annotations

import numpy as np

U32 = np.uint64(0xFFFFFFFF)


def philox4x32(ctr, key, rounds: int = 10):
    """Philox4x32 (Salmon et al. 2011): ctr [..., 4] and key [2] of 32-bit words
    in uint64 arrays; the output words [..., 4]."""
    c = [np.asarray(ctr[..., i], np.uint64) for i in range(4)]
    k0, k1 = int(key[0]), int(key[1])
    for _ in range(rounds):
        p0 = c[0] * np.uint64(0xD2511F53)
        p1 = c[2] * np.uint64(0xCD9E8D57)
        c = [(p1 >> np.uint64(32)) ^ c[1] ^ np.uint64(k0), p1 & U32,
             (p0 >> np.uint64(32)) ^ c[3] ^ np.uint64(k1), p0 & U32]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return np.stack(c, -1)


def threshold(p: float) -> int:
    """round(65536 p) of the fp32 value of p, ties to even."""
    return int(np.rint(np.float64(np.float32(p)) * 65536.0))


def scale(p: float) -> np.float32:
    t = threshold(p)
    return np.float32(0.0 if t == 65536 else 65536.0 / (65536 - t))


def keep_rows(rows, cols: int, p: float, seed: int, offset: int) -> np.ndarray:
    """Truth values [len(rows), cols] of the given rows of a [.][cols] tensor."""
    rows = np.asarray(rows, np.uint64)
    per = (cols + 7) // 8
    j = np.arange(cols)
    g = rows[:, None] * np.uint64(per) + np.arange(per, dtype=np.uint64)[None, :]
    ctr = np.stack([g & U32, g >> np.uint64(32), np.full_like(g, offset & 0xFFFFFFFF), np.full_like(g, offset >> 32)], -1)
    w = philox4x32(ctr, (seed & 0xFFFFFFFF, seed >> 32))
    word = w[:, j // 8, (j % 8) // 2]
    bits = (word >> (16 * (j % 2)).astype(np.uint64)) & np.uint64(0xFFFF)
    return bits >= np.uint64(threshold(p))


def keep(rows: int, cols: int, p: float, seed: int, offset: int) -> np.ndarray:
    return keep_rows(np.arange(rows), cols, p, seed, offset)


def dropout(x, p: float, seed: int, offset: int, res=None, rows=None) -> np.ndarray:
    """(res +) dropout(x) in float64, c in its exact value."""
    x = np.asarray(x, np.float64)
    k = keep_rows(np.arange(x.shape[0]) if rows is None else rows, x.shape[1], p, seed, offset)
    t = threshold(p)
    c = 0.0 if t == 65536 else 65536.0 / (65536 - t)
    y = np.where(k, x * c, 0.0)
    return y if res is None else np.asarray(res, np.float64) + y
