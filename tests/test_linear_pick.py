"""Which kernel sv_linear takes: the shapes that the GPU tests compare with a
reference reach every one of them, with operands of either type."""
import os
import re
import subprocess

from tests.linear_kernels import KERNELS, ROWS_16, ROWS_32

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "rejection_sampling_verify_09_amd", "csrc")

SOURCE = """
#include <cstdio>
#include "sv_linear_pick.hpp"
int main() {
  long long M, N, kbytes;
  std::printf("%d\\n", (int)(sizeof sv::kTiles / sizeof *sv::kTiles));
  while (std::scanf("%lld %lld %lld", &M, &N, &kbytes) == 3) std::printf("%d\\n", sv::pick_kernel(M, N, kbytes));
}
"""


def picks(tmp_path, shapes):
    src, exe = tmp_path / "pick.cpp", tmp_path / "pick"
    src.write_text(SOURCE)
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-Werror", "-I" + CSRC, str(src), "-o", str(exe)], check=True, timeout=120)
    r = subprocess.run([str(exe)], input="\n".join("%d %d %d" % s for s in shapes), capture_output=True, text=True, check=True)
    tiles, *out = [int(v) for v in r.stdout.split()]
    return tiles, out


def test_the_tested_shapes_reach_every_kernel(tmp_path):
    want, shapes = [], []
    for element in (2, 1):  # bytes of bfloat16 and e4m3
        for kernel, M, N, K in KERNELS:
            want.append(kernel)
            shapes.append((M, N, K * element))
    tiles, got = picks(tmp_path, shapes)
    assert got == want, [(s, g, w) for s, g, w in zip(shapes, got, want) if g != w]
    assert set(want) == {ROWS_16, ROWS_32, *range(tiles)}


def test_every_pick_is_launched():
    """The launch has a case for each tile of the table (the last one's is the default)."""
    with open(os.path.join(CSRC, "sv_linear.hip")) as f:
        text = f.read()
    cases = re.findall(r"(case -?\w+|default): return launch_(tile|rows)<MODE, OUT, ([\d, ]+)>", text)
    tiles = [[int(v) for v in args.split(",")] for _, kind, args in cases if kind == "tile"]
    with open(os.path.join(CSRC, "sv_linear_pick.hpp")) as f:
        table = re.findall(r"\{(\d+), (\d+), (\d+), \d+, [\d.]+f, [\d.]+f\}", f.read())
    # launch_tile<.., MB, NB, WM, WN, WK, D>: 16 MB WM rows, 16 NB WN columns, WK steps a round
    assert [(16 * t[0] * t[2], 16 * t[1] * t[3], t[4]) for t in tiles] == [tuple(int(v) for v in row) for row in table]
