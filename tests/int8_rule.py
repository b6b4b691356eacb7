"""The rule by which the 8-bit product takes its form, written a second time: which form and
how many K parts a shape gets, so that tests can name shapes on both sides of it."""
import numpy as np

F = np.float32
# path, weight rows, activation rows, us a round, us a round and 1000 k
TILES = (("large", 256, 256, 20.0, 10.0), ("wide", 256, 128, 12.0, 7.0), ("medium", 128, 128, 9.0, 4.6),
         ("small", 64, 128, 7.0, 3.5), ("narrow", 64, 64, 5.5, 2.6))


def few_block(N):
    per = 1
    while 8 * -(-N // (2048 * per)) > 32:
        per += 1
    return 8 * -(-N // (2048 * per))


def plan(M, N, K):
    """(path, parts); few rows: ("few", weight rows of a workgroup)."""
    best, least = None, F(np.inf)
    for path, tn, tm, start, per_k in TILES:
        tiles = -(-M // tm) * -(-N // tn)
        parts = 1
        while parts == 1 or parts <= min(256 // tiles, K // 512, 16):
            rounds, k = -(-tiles * parts // 256), -(-K // parts)
            busy = F(tiles * parts) / F(256 * rounds)
            us = F(rounds) * (F(start) + F(per_k) * F(1e-3) * F(k) * (F(0.8) + F(0.2) * busy))
            if parts > 1:
                us += F(2.5) + F(0.3) * (F(parts) + F(0.5)) * F(M * N) * F(4e-6)
            if us < least:
                least, best = us, (path, parts)
            parts += 1
    if M <= 16 and M * ((K + 111) // 128 * 128 + 16) <= 80 * 1024:
        rows = few_block(N)
        per_cu = -(-(-(-N // rows)) // 256)
        if F(3.0) + F(0.18e-6) * F(N * K) + F(0.04e-3) * F(M * K * per_cu) < least:
            best = ("few", rows)
    return best
