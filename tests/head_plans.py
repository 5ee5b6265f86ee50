"""Shapes of the vocabulary head that between them reach every tile shape and every way of sharing out rows,
each with the way the library cuts it up (`plan` reads that from the library's own planning header).

Entries: stats and gradz (the logits' products), store (grad_weight's): a tile shape, with "A+" or "B+" before it
where the first rows of that side go to 256 x 256 tiles; acc (grad_hidden's): tile shape, whether tiles are taken
whole, whether the others are shared by several workgroups; pieces of the vocabulary.
"""

import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "draft_verification_04_amd")

# (N, V, d, dtype): stats, gradz, store, acc, pieces
PLANS = {
    (61, 4500, 200, "bf16"): ("small", "small", "mid", ("thin", False, True), 1),
    (1, 1000, 4096, "bf16"): ("small", "small", "mid", ("thin", False, True), 1),
    (61, 45000, 200, "bf16"): ("thin", "thin", "big", ("thin", False, True), 1),
    (5, 300001, 16, "bf16"): ("thin", "thin", "mid", ("thin", False, True), 2),
    (40, 90000, 512, "bf16"): ("thin", "thin", "big", ("thin", False, True), 1),
    (348, 717, 3064, "bf16"): ("small", "small", "mid", ("mid", False, False), 1),
    (273, 4258, 408, "bf16"): ("deep", "deep", "mid", ("mid", False, True), 1),
    (67, 14497, 72, "bf16"): ("deep", "deep", "mid", ("mid", False, True), 1),
    (270, 4300, 448, "bf16"): ("deep", "deep", "mid", ("mid", False, True), 1),
    (8200, 700, 72, "bf16"): ("mid", "mid", "mid", ("mid", False, False), 1),
    (2048, 4000, 4352, "bf16"): ("mid", "mid", "A+mid", ("mid", True, True), 1),
    (4096, 2048, 4352, "bf16"): ("mid", "mid", "big", ("big", True, True), 1),
    (4096, 17000, 4352, "bf16"): ("A+mid", "A+mid", "B+mid", ("big", True, True), 2),
    (1025, 16500, 1000, "bf16"): ("A+mid", "A+mid", "B+mid", ("big", False, True), 1),
    (1025, 70001, 64, "bf16"): ("big", "big", "mid", ("mid", False, True), 2),
    (2100, 300, 1032, "f32"): ("small", "small", "small", ("small", True, True), 1),
    (2048, 4000, 4352, "f32"): ("thin", "thin", "thin", ("thin", True, True), 1),
    (5, 40001, 1000, "f32"): ("small", "thin", "thin", ("small", False, True), 2),
}

_MAIN = r"""
#include <stdio.h>
#include "xent_plan.hpp"
using namespace spec;
int main() {
  const char* name[] = {"big", "mid", "thin", "deep", "small"};
  int N, V, d, dtype;
  while (scanf("%d %d %d %d", &N, &V, &d, &dtype) == 4) {
    const int es = dtype == SPEC_BF16 ? 2 : 4;
    const BackPlan p = back_plan(N, V, d, dtype);
    auto show = [&](long long a, long long b, int kbytes, bool store) {
      const Shape s = pick_shape(a, b, kbytes, es, store);
      const bool split = s.head > 0 && (s.along_a || store);
      printf("%s%s ", split ? (s.along_a ? "A+" : "B+") : "", name[split || s.head == 0 ? s.tail : (int)kBig]);
    };
    show(V, N, d * es, false);
    show(V < p.vc ? V : p.vc, N, d * es, false);
    show(d, V < p.vc ? V : p.vc, (int)(p.npad * es), true);
    const long long tiles = (long long)ceil_div(d, tile_m(p.tile)) * ceil_div(N, tile_n(p.tile));
    printf("%s %d %d %d\n", name[p.tile], p.whole > 0, tiles > p.whole && p.parts > 1, p.pieces);
  }
}
"""


def plan(shapes, folder):
    """The library's plans of `shapes`, by compiling its planning header for the host."""
    src, exe = os.path.join(folder, "plan.cpp"), os.path.join(folder, "plan")
    with open(src, "w") as f:
        f.write(_MAIN)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), "-I",
                    os.path.join(PKG, "csrc"), src, "-o", exe], check=True, timeout=120)
    lines = "".join(f"{N} {V} {d} {int(t == 'bf16')}\n" for N, V, d, t in shapes)
    out = subprocess.run([exe], input=lines, capture_output=True, text=True, check=True, timeout=60).stdout
    res = []
    for line in out.splitlines():
        stats, gradz, store, tile, whole, shared, pieces = line.split()
        res.append((stats, gradz, store, (tile, whole == "1", shared == "1"), int(pieces)))
    return res
