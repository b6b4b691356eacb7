"""Which kernels the mixture-of-experts layer takes for a size (CPU): told by its workspace,
which for the few-token kernels holds rows of the second product for every pair."""
import os

import pytest


@pytest.fixture(scope="module")
def size():
    from weight_only_bit_amd import _lib, build
    if not os.path.exists(_lib.LIB_PATH):
        build.build()
    return _lib.lib()


def _up(n):
    return (n + 255) // 256 * 256


def _few(size, T, E, topk, H, I):
    """Units of 64 bytes and an id a pair, the activated rows, fp32 rows; else the choice and
    the activated rows, then the second stage's workspace."""
    P = T * topk
    few = _up(16 + 68 * P) + _up(2 * P * I) + 4 * P * H
    many = 2 * _up(4 * P) + _up(2 * P * I) + size.mxfp4_moe_stage2_workspace_size(T, topk, E, H, I)
    got = size.mxfp4_moe_layer_workspace_size(T, topk, E, H, I)
    assert few != many and got in (few, many)
    return got == few


@pytest.mark.parametrize("few,T,E,topk,H,I", [
    # the limits of the lists and of the staged rows
    (1, 64, 64, 8, 128, 64), (0, 65, 64, 2, 128, 64), (0, 57, 64, 9, 128, 64), (0, 9, 70, 64, 64, 64),
    (1, 5, 256, 6, 64, 128), (0, 5, 257, 6, 64, 128), (1, 8, 2, 2, 8448, 64), (0, 8, 2, 2, 8512, 64),
    (1, 8, 2, 2, 64, 8960), (0, 8, 2, 2, 64, 9024), (1, 1, 2, 1, 32768, 64), (0, 1, 2, 1, 32832, 64),
    # up to 8 tokens an expert is read once
    (1, 8, 64, 64, 128, 64), (1, 8, 8, 8, 7168, 2048), (1, 8, 32, 32, 64, 4096),
    # pairs: 256 or 10 an expert
    (1, 64, 4, 4, 2880, 2880), (1, 32, 8, 8, 2880, 2880), (0, 33, 8, 8, 2880, 2880), (0, 64, 16, 8, 2880, 2880),
    (1, 40, 32, 8, 2880, 2880), (0, 41, 32, 8, 2880, 2880), (0, 64, 32, 8, 2880, 2880), (1, 64, 64, 8, 2880, 2880),
    # rows that leave room for one or two workgroups on a CU: 96, or 4 an expert
    (1, 48, 8, 2, 4096, 64), (0, 49, 8, 2, 4096, 64), (1, 64, 64, 4, 4096, 1792), (0, 33, 64, 8, 4096, 1792),
    (1, 32, 32, 4, 2048, 7168), (0, 33, 32, 4, 2048, 7168), (0, 64, 16, 4, 4096, 1792), (0, 64, 64, 8, 7168, 2048)])
def test_kernels_for_few_tokens_by_pairs_and_rows(size, few, T, E, topk, H, I):
    assert _few(size, T, E, topk, H, I) == bool(few)
