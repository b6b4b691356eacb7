"""The forms of the MXFP4 product's tiles and of the layer's products that are built,
and the tiles' hand-counted waits (CPU: compiles to gfx950 assembly).

Every form that is built is reached by some call: the lists below hold one for
each, and nothing else is in the assembly.

Waits: a tile copies its operands into LDS (`global_load_lds`, which the compiler
does not count) group by group, up to NG groups ahead, and a barrier lets a group be
read.  The barrier at the end of group g needs group g + 1 in LDS, while the copies of
g + 2 .. g + NG - 1 stay in flight.  Between two barriers the copies of exactly one
group are started, and vector-memory operations complete in the order of issue, so
`s_waitcnt vmcnt(N)` before a barrier is enough if N is at most the number of copies
started in the NG - 2 stretches before it."""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "weight_only_bit_amd", "csrc")
HIPCC = shutil.which("hipcc") or ("/opt/rocm/bin/hipcc" if os.path.exists("/opt/rocm/bin/hipcc") else None)
needs_hipcc = pytest.mark.skipif(HIPCC is None, reason="hipcc not found")

# mxfp4_tile_kernel: (weight rows, activation rows, scales) -> M, N, K
TILES = {
    (256, 256, "packed"): (2048, 8704, 64),
    (128, 128, "straight"): (1000, 1096, 6144),
    (128, 128, "whole"): (1000, 2104, 8160),       # 16 spans: the most that fit
    (128, 128, "packed"): (1000, 2104, 8224),      # 17
    (64, 128, "straight"): (100, 256, 128),
    (64, 128, "whole"): (100, 264, 352),
    (64, 64, "straight"): (40, 72, 5376),
    (64, 64, "whole"): (17, 72, 453664),           # 56 spans a part: the most that fit
    (64, 64, "packed"): (17, 72, 475168),          # 59
}
# moe_few_kernel: (up, one token, scores a lane, waves, groups, steps) -> T, E, topk, H, I
FEW = {
    (1, 1, 2, 8, 1, 2): (1, 32, 4, 2048, 64), (1, 1, 2, 8, 1, 3): (1, 32, 4, 2112, 64),
    (1, 1, 16, 8, 1, 2): (1, 33, 4, 2048, 64), (1, 1, 16, 8, 1, 3): (1, 33, 4, 2112, 64),
    (1, 0, 1, 8, 1, 2): (8, 8, 2, 2048, 64), (1, 0, 1, 8, 1, 3): (8, 8, 2, 2112, 64),
    (1, 0, 1, 4, 2, 2): (9, 8, 2, 1024, 64), (1, 0, 1, 4, 2, 3): (9, 8, 2, 1088, 64),
    (0, 0, 1, 8, 1, 2): (4, 40, 35, 128, 1792), (0, 0, 1, 8, 1, 3): (5, 8, 2, 64, 2112),
    (0, 0, 1, 4, 2, 2): (9, 8, 2, 64, 1024), (0, 0, 1, 4, 2, 3): (9, 8, 2, 64, 1088),
}
SCALES = ("straight", "packed", "whole")


@pytest.fixture(scope="module")
def assembly(tmp_path_factory):
    flags = ["--offload-arch=gfx950", "-O3", "-std=c++17", "-Xclang", "-target-feature", "-Xclang",
             "-packed-fp32-ops", "-I", os.path.join(ROOT, "include"), "-I", CSRC,
             "--cuda-device-only", "-S"]
    td = tmp_path_factory.mktemp("asm")
    procs = {}
    for src in ("mx_gemm.hip", "moe_layer.hip"):
        out = str(td / (src + ".s"))
        procs[src] = (out, subprocess.Popen([HIPCC] + flags + ["-o", out, os.path.join(CSRC, src)],
                                            stdout=subprocess.PIPE, stderr=subprocess.STDOUT))
    texts = {}
    for src, (out, p) in procs.items():
        log = p.communicate(timeout=600)[0].decode(errors="replace")
        assert p.returncode == 0, log[-2000:]
        texts[src] = open(out).read()
    return texts


TILE = re.compile(r"^\S*mxfp4_tile_kernelINS0_6MxTileILi(\d+)ELi(\d+)ELi(\d+)ELi(\d+)ELi(\d+)EEE"
                  r"LNS0_6ScalesE(\d)E\S*:\s*;", re.M)
LAYER = re.compile(r"^\S*moe_few_kernelILb(\d)ELb(\d)ELi(\d+)ELi(\d+)ELi(\d+)ELi(\d+)E\S*:\s*;", re.M)


def tile_forms(text):
    """{(weight rows, activation rows, scales)}: WN waves of NB x MB blocks of 32 along n, 4 / WN along m."""
    return {(32 * nb * wn, 32 * mb * (4 // wn), SCALES[sc])
            for wn, nb, mb, _, _, sc in (tuple(map(int, m.groups())) for m in TILE.finditer(text))}


@needs_hipcc
def test_tile_forms_are_those_that_calls_reach(assembly):
    assert tile_forms(assembly["mx_gemm.hip"]) == set(TILES)


@needs_hipcc
def test_layer_forms_are_those_that_calls_reach(assembly):
    assert {tuple(map(int, m.groups())) for m in LAYER.finditer(assembly["moe_layer.hip"])} == set(FEW)


def tile_events(body):
    """Copies ("code" 16 bytes a lane, "word" 4), waits ("wait", N), "barrier", labels and
    branches back of one kernel, in order."""
    out = []
    for line in body.split("\n"):
        t = line.strip()
        if t.startswith("global_load_lds_dwordx4"):
            out.append(("code",))
        elif t.startswith("global_load_lds"):
            out.append(("word",))
        elif t.startswith("s_waitcnt") and "vmcnt" in t:
            out.append(("wait", int(re.search(r"vmcnt\((\d+)\)", t).group(1))))
        elif t.startswith("s_barrier"):
            out.append(("barrier",))
        elif re.match(r"\.LBB\w+:", t):
            out.append(("label", t.split(":")[0]))
        elif re.match(r"s_c?branch", t):
            out.append(("branch", t.split()[-1]))
    return out


def main_loop(events):
    """(first, past the last) event of the loop that holds the barriers: back to the label
    before it, without another label between."""
    label, found = (0, None), []
    for i, e in enumerate(events):
        if e[0] == "label":
            label = (i, e[1])
        elif e[0] == "branch" and e[1] == label[1] and ("barrier",) in events[label[0]:i]:
            found.append((label[0], i))
    assert len(found) == 1, found
    return found[0]


def waits_of(events):
    """[(N, copies since the barrier before)] for every barrier of a straight run of events."""
    out, since, wait = [], 0, None
    for e in events:
        if e[0] in ("code", "word"):
            since, wait = since + 1, None
        elif e[0] == "wait":
            wait = e[1]
        elif e[0] == "barrier":
            assert wait is not None, "a barrier without a wait of its own"
            out.append((wait, since))
            since, wait = 0, None
    return out, since


def first_scale(gs):
    """The stretch with the next span's scales, which start in the span's second step: with
    groups of one stage (two steps) that step follows the first barrier."""
    return 1 if gs == 1 else 0


def tile_faults(body, wn, nb, mb, gs, ng, scales):
    """What is wrong with a tile kernel's waits, as a list of texts."""
    rows, faults = 32 * nb * wn + 32 * mb * (4 // wn), []
    group = rows * 64 * gs // 4096                      # copies of a wave and group
    scale = {"whole": 0, "packed": (rows + 255) // 256, "straight": rows // 64}[scales]
    events = tile_events(body)
    first, last = main_loop(events)
    before, _ = waits_of([e for e in events[:first] if e[0] != "branch"])
    if len(before) != 1:
        return ["%d barriers before the loop" % len(before)]
    wait, issued = before[0]                            # the first scales, then group 0, come first
    if wait > issued - scale - group:
        faults.append("first wait %d of %d copies" % (wait, issued))
    spans, rest = waits_of(events[first:last])
    per = 4 // gs
    if len(spans) != per:
        return faults + ["%d barriers a span" % len(spans)]
    # copies of each stretch that ends in a barrier, round the loop
    stretch = [n + (rest if i == 0 else 0) for i, (_, n) in enumerate(spans)]
    for i, (wait, _) in enumerate(spans):
        if wait > sum(stretch[(i - k) % per] for k in range(ng - 2)):
            faults.append("barrier %d waits for all but %d, stretches %s" % (i, wait, stretch))
        if stretch[i] != group + (scale if i == first_scale(gs) else 0):
            faults.append("%d copies before barrier %d" % (stretch[i], i))
    if scale and per - 1 - first_scale(gs) < ng - 2:    # read after the span's last barrier
        faults.append("scales not landed at the span's last barrier")
    after, _ = waits_of(events[last:])
    if any(n for n, _ in after) or not after:
        faults.append("waits after the loop: %s" % after)
    return faults


@needs_hipcc
def test_tiles_wait_for_the_group_they_read_next(assembly):
    text = assembly["mx_gemm.hip"]
    seen = 0
    for m in TILE.finditer(text):
        *geometry, sc = map(int, m.groups())
        body = text[m.end():text.index(".Lfunc_end", m.end())]
        assert tile_faults(body, *geometry, SCALES[sc]) == [], m.group(0)
        # the check sees a wait that lets one copy more stay in flight
        loop = re.search(r"s_waitcnt vmcnt\((%d)\)[^\n]*\n(?:[^\n]*\n){0,3}\s*s_barrier" %
                         ((geometry[4] - 2) * (64 * geometry[3] * (32 * geometry[1] * geometry[0] + 32 * geometry[2]
                                                                  * (4 // geometry[0])) // 4096)), body)
        late = body[:loop.start(1)] + str(int(loop.group(1)) + 1) + body[loop.end(1):]
        assert tile_faults(late, *geometry, SCALES[sc])
        seen += 1
    assert seen == len(TILES)
