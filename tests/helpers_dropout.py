"""Dropout's random bits in numpy: Philox4x32 with ten rounds (Salmon, Moraes,
Dror and Shaw, 2011), from its definition."""
import numpy as np

LOW = np.uint64(0xFFFFFFFF)


def philox(counter, k0, k1):
    """counter: uint64 [4, n] of 32-bit words; four uint64 arrays of 32-bit words."""
    c = [w.astype(np.uint64) for w in counter]
    for r in range(10):
        a = np.uint64((k0 + r * 0x9E3779B9) & 0xFFFFFFFF)
        b = np.uint64((k1 + r * 0xBB67AE85) & 0xFFFFFFFF)
        p0, p1 = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)  # 32 x 32 bits: exact in 64
        c = [(p1 >> np.uint64(32)) ^ c[1] ^ a, p1 & LOW, (p0 >> np.uint64(32)) ^ c[3] ^ b, p0 & LOW]
    return c


def kept(first, count, p, seed, offset):
    """Which of `count` values from the first-th on (a multiple of 8) stay, and the factor of those that do."""
    at = np.arange(first // 8, (first + count + 7) // 8, dtype=np.uint64)
    counter = [at & LOW, at >> np.uint64(32), np.full_like(at, offset & 0xFFFFFFFF), np.full_like(at, offset >> 32)]
    words = philox(counter, seed & 0xFFFFFFFF, seed >> 32)
    bits = np.stack([w >> np.uint64(s) & np.uint64(0xFFFF) for w in words for s in (0, 16)], 1).reshape(-1)[:count]
    drop = round(p * 65536)
    return bits >= drop, 65536 / (65536 - drop) if drop < 65536 else 0.0
