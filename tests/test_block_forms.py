"""The forms of the 8-bit product, of the group-limited choice and of the row kernels that are
built, and the product tiles' hand-counted waits (CPU: compiles to gfx950 assembly).

Every form that is built is reached by some call, and nothing else is in the assembly.

Waits: a tile copies half groups (a group's weight rows, its activation rows) into a ring of
NH places in LDS (`global_load_lds`, which the compiler does not count).  The barrier at the
end of group g needs group g + 1 in LDS, while the NH - 4 halves behind it may be in flight.
Between two barriers the copies of exactly two halves are started, in the order of their use,
and vector-memory operations complete in the order of issue, so `s_waitcnt vmcnt(N)` before
the barrier is enough if N is at most the copies of NH - 4 halves."""
import os
import re
import subprocess

import pytest

from tests.test_kernel_forms import CSRC, HIPCC, ROOT, main_loop, needs_hipcc, tile_events, waits_of

# waves along n, blocks, stages of a group, half groups of the ring, nontemporal weights
TILES = {(2, 4, 4, 2, 5, 0), (4, 2, 4, 2, 6, 0)} | {(2, *t, nt) for t in ((2, 2, 2, 9), (1, 2, 2, 10), (1, 1, 2, 11))
                                                    for nt in (0, 1)}
FEW = {(4, 1, 0), (8, 1, 0), (2, 4, 0), (8, 1, 1), (4, 2, 1)}
F16, BF16, F32 = 0, 1, 3
TYPES = (F16, BF16, F32)
# threads of a row, pieces of eight elements a thread -> a row's length that takes them
NORM = {(8, 1): 64, (16, 1): 128, (32, 1): 256, (64, 1): 512, (64, 2): 1024, (256, 1): 2048,
        (512, 1): 4096, (512, 2): 8192, (1024, 2): 16384, (1024, 4): 32768}
ROWS8 = {(8, 1): 64, (16, 1): 128, (32, 1): 256, (64, 1): 512, (64, 2): 1024, (256, 1): 2048,
         (256, 2): 4096, (512, 2): 8192, (512, 4): 16384, (512, 6): 24576, (1024, 4): 32768, (1024, 8): 65536}


@pytest.fixture(scope="module")
def assembly(tmp_path_factory):
    flags = ["--offload-arch=gfx950", "-O3", "-std=c++17", "-Xclang", "-target-feature", "-Xclang",
             "-packed-fp32-ops", "-I", os.path.join(ROOT, "include"), "-I", CSRC, "--cuda-device-only", "-S"]
    td = tmp_path_factory.mktemp("asm")
    procs = {}
    for src in ("int8_gemm.hip", "int8_quant.hip", "residual_norm.hip", "moe_route.hip"):
        out = str(td / (src + ".s"))
        procs[src] = (out, subprocess.Popen([HIPCC] + flags + ["-o", out, os.path.join(CSRC, src)],
                                            stdout=subprocess.PIPE, stderr=subprocess.STDOUT))
    texts = {}
    for src, (out, p) in procs.items():
        log = p.communicate(timeout=600)[0].decode(errors="replace")
        assert p.returncode == 0, log[-2000:]
        texts[src] = open(out).read()
    return texts


def forms(text, kernel, count):
    """The template arguments of every instance of a kernel."""
    pattern = r"^\S*%s\S*?I%s" % (kernel, r"\D*?L[ib](\d+)E" * count)
    return {tuple(map(int, m.groups())) for m in re.finditer(pattern + r"\S*:\s*;", text, re.M)}


TILE = re.compile(r"^\S*int8_tile_kernelINS0_8Int8TileILi(\d+)ELi(\d+)ELi(\d+)ELi(\d+)ELi(\d+)EEELb([01])EE\S*:\s*;", re.M)


@needs_hipcc
def test_product_forms(assembly):
    text = assembly["int8_gemm.hip"]
    assert {tuple(map(int, m.groups())) for m in TILE.finditer(text)} == TILES
    assert forms(text, "int8_few_kernel", 3) == FEW


@needs_hipcc
def test_row_forms(assembly):
    types = {(t, r) for t in TYPES for r in (t, F32)}
    assert forms(assembly["residual_norm.hip"], "residual_norm_kernel", 4) == {t + s for t in types for s in NORM}
    assert forms(assembly["int8_quant.hip"], "int8_quantize_kernel", 4) == {
        (t, act) + s for t in TYPES for act in (0, 1) for s in ROWS8}
    assert forms(assembly["int8_quant.hip"], "int8_dequant_kernel", 1) == {(t,) for t in TYPES}


def route_form(T, E, groups):
    """(lanes, registers, quads) of the choice for T tokens of E experts."""
    size = E // groups

    def split(lanes):
        span = 1
        while 2 * span * groups <= lanes:
            span *= 2
        run = -(-size // span)
        return -(-run // 4) * 4 if size % 4 == 0 else run
    lanes = 16 if groups <= 16 and split(16) <= (4 if T <= 2048 else 16) else 64
    V = 2
    while V < split(lanes):
        V *= 2
    return lanes, V, int(V % 4 == 0 and size % 4 == 0)


@needs_hipcc
def test_route_forms(assembly):
    reached = {route_form(T, E, g) for T in (1, 4096) for E in range(1, 1025) for g in range(1, 65) if E % g == 0}
    assert max(v for _, v, _ in reached) == 32
    assert forms(assembly["moe_route.hip"], "moe_route_kernel", 4) == {(t,) + f for t in TYPES for f in reached}


def tile_faults(body, wn, nb, mb, gs, nh, nt):
    """What is wrong with a tile kernel's waits, as a list of texts."""
    copies = (32 * nb * wn + 32 * mb * (4 // wn)) * 64 * gs // 4096  # of a wave and group
    faults, events = [], tile_events(body)
    first, last = main_loop(events)
    before, _ = waits_of([e for e in events[:first] if e[0] != "branch"])
    if len(before) != 1:
        return ["%d barriers before the loop" % len(before)]
    wait, issued = before[0]  # group 0 comes first
    if wait > issued - copies:
        faults.append("first wait %d of %d copies" % (wait, issued))
    rounds, rest = waits_of(events[first:last])
    if len(rounds) != 1:
        return faults + ["%d barriers a group" % len(rounds)]
    wait, since = rounds[0]
    if since + rest != copies:
        faults.append("%d copies a group" % (since + rest))
    if wait > (nh - 4) * copies // 2:
        faults.append("a wait for all but %d" % wait)
    # behind it no copy is started, and none is in flight when the ring becomes staging space
    after = events[last:]
    waits = [e[1] for e in after[:after.index(("barrier",))] if e[0] == "wait"]
    if any(e[0] in ("code", "word") for e in after) or not waits or waits[-1] != 0:
        faults.append("copies or waits after the loop: %s" % after)
    return faults


@needs_hipcc
def test_tiles_wait_for_the_group_they_read_next(assembly):
    text, seen = assembly["int8_gemm.hip"], 0
    for m in TILE.finditer(text):
        wn, nb, mb, gs, nh, _ = geometry = tuple(map(int, m.groups()))
        body = text[m.end():text.index(".Lfunc_end", m.end())]
        assert tile_faults(body, *geometry) == [], geometry
        # the check sees a wait that lets one copy more stay in flight
        n = (nh - 4) * (32 * nb * wn + 32 * mb * (4 // wn)) * 64 * gs // 8192
        loop = re.search(r"s_waitcnt vmcnt\((%d)\)[^\n]*\n(?:[^\n]*\n){0,3}\s*s_barrier" % n, body)
        late = body[:loop.start(1)] + str(n + 1) + body[loop.end(1):]
        assert tile_faults(late, *geometry)
        seen += 1
    assert seen == len(TILES)


@needs_hipcc
def test_no_tile_loop_touches_scratch(assembly):
    text = assembly["int8_gemm.hip"]
    for m in TILE.finditer(text):
        body = text[m.end():text.index(".Lfunc_end", m.end())]
        assert "scratch_" not in body, m.group(0)
