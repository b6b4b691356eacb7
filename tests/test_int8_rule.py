"""The 8-bit product's choice of form (CPU): the rule written a second time gives the K parts
that the library's workspace sizes show, and every form that is built is reached."""
import os
import random

import pytest

from tests.int8_rule import few_block, few_form, plan


@pytest.fixture(scope="module")
def L():
    from weight_only_bit_amd import _lib, build
    if not os.path.exists(_lib.LIB_PATH):
        build.build()
    return _lib


def test_parts_are_those_of_the_workspace(L):
    r = random.Random(3)
    paths = set()
    for _ in range(20000):
        M, N, K = int(2 ** r.uniform(0, 12)), 8 * int(2 ** r.uniform(0, 12)), 16 * int(2 ** r.uniform(0, 13))
        if K > 131056 or M * K >= 2 ** 32 or N * K >= 2 ** 32:
            continue
        path, parts = plan(M, N, K)
        paths.add((path, path != "few" and parts > 1))
        want = 0 if path == "few" or parts == 1 else parts * M * N * 4
        assert L.lib().int8_gemm_workspace_size(M, N, K) == want, (M, N, K)
    assert paths == {("few", False)} | {(p, s) for p in ("large", "wide", "medium", "small", "narrow")
                                        for s in (False, True)}


def test_a_part_has_a_group_at_least():
    for K in (16, 496, 512, 1024, 8192, 131056):
        for M, N in ((17, 8), (1, 64), (100, 64), (2000, 8)):
            path, parts = plan(M, N, K)
            assert path == "few" or parts <= max(1, -(-K // 128))


def test_few_rows_blocks():
    for N in (8, 16, 2048, 2056, 4096, 4104, 5376, 6144, 8192, 8200, 16384, 43008, 131072):
        for M in (1, 2, 3, 8, 9, 16):
            for K in (16, 4096, 4112):
                rows, (_, groups) = few_block(M, N, K), few_form(M, N, K)
                assert rows % 8 == 0 and 8 <= rows <= groups * (16 if M > 8 else 8) <= 32
    assert [few_block(4, N, 5376) for N in (2048, 4096, 5376, 5760, 16384)] == [8, 8, 24, 24, 32]
    assert [few_block(13, N, 2880) for N in (2048, 4096, 5376, 5760, 16384)] == [8, 16, 24, 24, 32]
    assert few_block(1, 16384, 5376) == 8
