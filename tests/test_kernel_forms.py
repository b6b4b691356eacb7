"""The forms of the MXFP4 product's tiles and of the layer's products that are built
(CPU: compiles to gfx950 assembly).

Every form that is built is reached by some call: the lists below hold one for
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
