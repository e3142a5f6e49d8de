"""The counter-based keep mask of LoRA dropout (oracle -- test infrastructure
only): Philox4x32 with 7 rounds, from its definition (J. Salmon, M. Moraes,
R. Dror and D. Shaw, "Parallel random numbers: as easy as 1, 2, 3", SC 2011),
in Python integers.

Key = the 64-bit seed; counter = (column // 8, row, offset low, offset high).
16-bit half i of the four output words (low half of the first word first)
decides column 8 (column // 8) + i: dropped when it is below
T = round(65536 p), at most 65535.
"""

from __future__ import annotations

import numpy as np

M0, M1 = 0xD2511F53, 0xCD9E8D57
W0, W1 = 0x9E3779B9, 0xBB67AE85
MASK = 0xFFFFFFFF


def philox4x32(counter, key, rounds: int):
    c0, c1, c2, c3 = counter
    k0, k1 = key
    for _ in range(rounds):
        p0, p1 = M0 * c0, M1 * c2
        c0, c1, c2, c3 = (p1 >> 32) ^ c1 ^ k0, p1 & MASK, (p0 >> 32) ^ c3 ^ k1, p0 & MASK
        k0, k1 = (k0 + W0) & MASK, (k1 + W1) & MASK
    return c0, c1, c2, c3


def threshold(p: float) -> int:
    return min(65535, round(p * 65536))


def keep_mask(seed: int, offset: int, p: float, M: int, n: int) -> np.ndarray:
    """bool [M, n]; seed and offset as 64-bit patterns (negative ones wrap)."""
    seed, offset = seed & (2 ** 64 - 1), offset & (2 ** 64 - 1)
    T = threshold(p)
    out = np.zeros((M, n), dtype=bool)
    for m in range(M):
        for g in range(n // 8):
            w = philox4x32((g, m, offset & MASK, offset >> 32), (seed & MASK, seed >> 32), 7)
            for i in range(8):
                out[m, 8 * g + i] = ((w[i // 2] >> (16 * (i % 2))) & 0xFFFF) >= T
    return out
