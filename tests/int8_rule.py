"""The rule by which the 8-bit product takes its form, written a second time: which form and
how many K parts a shape gets, so that tests can name shapes on both sides of it."""
import numpy as np

F = np.float32
# path, weight rows, activation rows, us a round, us a round and 1000 k, us a million bytes of weights
TILES = (("large", 256, 256, 7.9, 13.0, 0.24), ("wide", 256, 128, 6.2, 7.9, 0.21), ("medium", 128, 128, 5.4, 5.1, 0.19),
         ("small", 64, 128, 4.6, 3.6, 0.17), ("narrow", 64, 64, 3.4, 2.4, 0.17))


def few_form(M, N, K):
    """(waves that share rows, groups of rows) of a workgroup"""
    if M > 8:
        return (8, 1) if N <= 4096 else (4, 2)
    if N <= 4096:
        return 4, 1
    return (8, 1) if M <= 2 and N > 8192 and K >= 5120 else (2, 4)


def few_block(M, N, K):
    per = 1
    while 8 * -(-N // (2048 * per)) > 32:
        per += 1
    return min(8 * -(-N // (2048 * per)), few_form(M, N, K)[1] * (16 if M > 8 else 8))


def plan(M, N, K):
    """(path, parts); few rows: ("few", weight rows of a workgroup)."""
    best, least = None, F(np.inf)
    for path, tn, tm, start, per_k, per_mb in TILES:
        tiles = -(-M // tm) * -(-N // tn)
        parts = 1
        while parts == 1 or parts <= min(256 // tiles, K // 512, 16):
            rounds, k = -(-tiles * parts // 256), -(-K // parts)
            busy = F(tiles * parts) / F(256 * rounds)
            us = F(rounds) * F(start) + max(F(rounds) * F(per_k) * F(1e-3) * F(k) * (F(0.65) + F(0.35) * busy),
                                            F(per_mb) * F(1e-6) * F(N * K))
            if parts > 1:
                us += F(1.8) + F(0.33) * (F(parts) + F(0.5)) * F(M * N) * F(4e-6)
            if us < least:
                least, best = us, (path, parts)
            parts += 1
    if M <= 16 and M * ((K + 111) // 128 * 128 + 16) <= 80 * 1024:
        rows = few_block(M, N, K)
        per_cu = -(-(-(-N // rows)) // 256)
        stage = F(0.005e-3) if M <= 8 and rows == 8 and N > 8192 else F(0.035e-3)
        if F(2.8) + F(0.17e-6) * F(N * K) + stage * F(M * K * per_cu) < least:
            best = ("few", rows)
    return best
