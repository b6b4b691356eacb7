"""What the assembly of the 8-bit product, the row kernels and the group-limited choice shows beyond the
tiles' waits (CPU: compiles to gfx950 assembly)."""
import re

from tests.test_block_forms import TILE, TILES, assembly, needs_hipcc  # noqa: F401 (a fixture)


def copies(wn, nb, mb, gs, nh):
    """Copies of a wave by their places: (weights that fill the ring at the start, weights after that,
    activations).  The ring's halves but the last two are filled, and a step's share of the next group;
    the loop copies a group."""
    weights, rows = 32 * nb * wn, 32 * mb * (4 // wn)
    a, b = weights * 64 * gs // 4096, rows * 64 * gs // 4096  # of a group
    step = (a + b) // (2 * gs)
    if nh % 2:  # halves of one size; the place that is free first is one of activation rows
        assert a == b
        return (nh - 1) // 2 * a, a, (nh - 3) // 2 * b + step + b
    assert step <= a
    return (nh // 2 - 1) * a, step + a, (nh // 2 - 1) * b + b


@needs_hipcc
def test_weight_copies_after_the_first_are_nontemporal(assembly):  # noqa: F811
    text, seen = assembly["int8_gemm.hip"], 0
    for m in TILE.finditer(text):
        *tile, nt = map(int, m.groups())
        body = text[m.end():text.index(".Lfunc_end", m.end())]
        lines = re.findall(r"global_load_lds_dwordx4.*", body)
        marked = sum(bool(re.search(r"\bnt\b", line)) for line in lines)
        first, later, rows = copies(*tile)
        assert len(lines) == first + later + rows and marked == (later if nt else 0), tile
        seen += 1
    assert seen == len(TILES)


@needs_hipcc
def test_no_kernel_keeps_a_row_in_scratch_memory(assembly):  # noqa: F811
    for src, text in assembly.items():
        kernels = re.findall(r"^; Kernel info:.*?^; ScratchSize: (\d+)", text, re.M | re.S)
        assert kernels and len(kernels) == text.count(".amdhsa_kernel "), src
        assert all(size == "0" for size in kernels) and "scratch_" not in text, src
