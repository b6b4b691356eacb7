"""The forms of the MXFP4 product's tiles that are built (CPU: compiles to gfx950
assembly).

Every form that is built is reached by some call: the list below holds one for
each, and nothing else is in the assembly."""
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
SCALES = ("straight", "packed", "whole")


@pytest.fixture(scope="module")
def assembly(tmp_path_factory):
    flags = ["--offload-arch=gfx950", "-O3", "-std=c++17", "-Xclang", "-target-feature", "-Xclang",
             "-packed-fp32-ops", "-I", os.path.join(ROOT, "include"), "-I", CSRC,
             "--cuda-device-only", "-S"]
    td = tmp_path_factory.mktemp("asm")
    procs = {}
    for src in ("mx_gemm.hip",):
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


def tile_forms(text):
    """{(weight rows, activation rows, scales)}: WN waves of NB x MB blocks of 32 along n, 4 / WN along m."""
    return {(32 * nb * wn, 32 * mb * (4 // wn), SCALES[sc])
            for wn, nb, mb, _, _, sc in (tuple(map(int, m.groups())) for m in TILE.finditer(text))}


@needs_hipcc
def test_tile_forms_are_those_that_calls_reach(assembly):
    assert tile_forms(assembly["mx_gemm.hip"]) == set(TILES)
