"""The 8-bit product's workspace size is 0 for every shape that the product refuses, so that a refused
call takes no memory for it (CPU)."""
import random

import pytest

from tests.test_block_abi import F, L, wob  # noqa: F401 (fixtures)


def refused(M, N, K):
    return (K % 16 != 0 or N % 8 != 0 or not 16 <= K <= 131056 or M < 0 or N < 0 or M * K >= 2 ** 32 or N * K >= 2 ** 32
            or M >= 2 ** 27 or N >= 2 ** 27)


def status(lib, M, N, K):
    return lib.int8_gemm(F.p, F.p, F.p, F.p, None, F.odd, 1, M, N, K, None, 0, None)


@pytest.mark.parametrize("M,N,K", [(100, 5376, 21500), (100, 5378, 21504), (100, 5376, 21512), (100, 5376, 131072),
                                   (-1, 5376, 21504), (100, -8, 21504), (100, 5376, 8), (100, 65544, 65536),
                                   (65536, 8, 65536), (100, 199736, 21504), (1 << 27, 8, 16)])
def test_refused_shapes_need_nothing(L, M, N, K):  # noqa: F811
    assert refused(M, N, K) and status(L.lib(), M, N, K) == L.INVALID_ARG
    assert L.lib().int8_gemm_workspace_size(M, N, K) == 0


def test_shapes_next_to_the_limits(L):  # noqa: F811
    """Random shapes on both sides: the size is 0 on the refused ones, and a product that is taken asks for what
    the size says."""
    r, seen = random.Random(4), set()
    for _ in range(4000):
        M, N, K = int(2 ** r.uniform(0, 21)), int(2 ** r.uniform(3, 21)), int(2 ** r.uniform(4, 17.2))
        if r.random() < 0.8:
            N, K = -(-N // 8) * 8, -(-K // 16) * 16
        bad = refused(M, N, K)
        size = L.lib().int8_gemm_workspace_size(M, N, K)
        assert not (bad and size)
        seen.add((bad, size > 0))
    assert seen == {(True, False), (False, False), (False, True)}


def test_binding_sees_the_same(L, wob):  # noqa: F811
    wob.int8_gemm_workspace_size.cache_clear()
    assert wob.int8_gemm_workspace_size(100, 5378, 21504) == 0
    assert wob.int8_gemm_workspace_size(100, 5376, 21504) > 0
