"""Shapes of the 8-bit head's product by the tile that the library picks for them (`plan` reads that from the library's
own planning header), for the GPU tests: rows and vocabularies that end inside a tile, last blocks of k that are whole
and cut, fewer blocks than the pipeline has stages."""

import os
import subprocess

from conftest import ROOT

PKG = os.path.join(ROOT, "draft_verification_04_amd")
TILES = ["256x256", "256x128", "128x128", "128x64", "128x32", "64x64", "64x32"]

# (rows, vocabulary, width): tile for bf16 and for fp32 logits
PLANS = {
    (600, 40007, 128): ("256x256", "128x128"),
    (513, 65001, 400): ("256x256", "128x128"),
    (200, 40001, 272): ("256x256", "128x128"),
    (300, 20011, 1040): ("256x128", "128x128"),
    (200, 20011, 2064): ("256x128", "128x128"),
    (700, 30001, 144): ("128x128", "128x128"),
    (200, 9001, 272): ("128x128", "128x128"),
    (64, 65001, 400): ("128x64", "128x64"),
    (50, 40001, 128): ("128x64", "128x64"),
    (32, 151936, 128): ("128x32", "128x32"),
    (20, 20011, 1040): ("128x32", "128x32"),
    (50, 9001, 272): ("64x64", "64x64"),
    (50, 9001, 128): ("64x64", "64x64"),
    (100, 3001, 2064): ("64x32", "64x32"),
    (65, 1003, 144): ("64x32", "64x32"),
    (3, 1003, 272): ("64x32", "64x32"),
}

_MAIN = r"""
#include <cstdio>
#include "logits_plan.hpp"
int main() {
  int N, V, d;
  while (std::scanf("%d %d %d", &N, &V, &d) == 3)
    std::printf("%d %d\n", spec::pick_logit_tile(false, N, V, d), spec::pick_logit_tile(true, N, V, d));
}
"""


def plan(shapes, folder):
    """The library's tiles for `shapes`, by compiling its planning header for the host."""
    src, exe = os.path.join(folder, "tiles.cpp"), os.path.join(folder, "tiles")
    with open(src, "w") as f:
        f.write(_MAIN)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), "-I",
                    os.path.join(PKG, "csrc"), src, "-o", exe], check=True, timeout=120)
    out = subprocess.run([exe], input="".join("%d %d %d\n" % s for s in shapes), capture_output=True, text=True, check=True,
                         timeout=60).stdout
    return [tuple(TILES[int(t)] for t in line.split()) for line in out.splitlines()]
