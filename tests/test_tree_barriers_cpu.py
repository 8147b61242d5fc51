"""The barriers of the tree attention kernels, walked on the CPU with the kernels'
own ring sizes (csrc/tree_rings.h) in every order that holding one warp, copy or
MMA back gives: no wait by parity takes one phase for another, and no stage is
read before its tile is there (no GPU needed)."""
import json
import os
import subprocess

import pytest

import _ring_model as model

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "swiglu_block_quantized_gb300", "csrc")

# runs of one CTA: (tiles, masked ones at its end)
RUNS = [[(12, 1)], [(1, 1), (1, 1), (2, 1), (7, 3), (1, 0)], [(3, 0), (4, 4), (5, 2)]]

PRINT_FEW = """
#include <cstdio>
#include "tree_rings.h"
using namespace m4q;
int main() {
  const char* sep = "[";
  for (int d = 64; d <= 128; d += 64)
    for (int q8 = 0; q8 < 2; ++q8)
      for (int nc = 1; nc <= 2; ++nc) {
        const FewRings r = few_rings(d, q8 != 0, nc);
        std::printf("%s{\\"d\\": %d, \\"q8\\": %d, \\"nc\\": %d, \\"ks\\": %d, \\"vs\\": %d, \\"rs\\": %d, \\"groups\\": %d, "
                    "\\"ok\\": %d, \\"raw_bar\\": [", sep, d, q8, nc, r.ks, r.vs, r.rs, r.groups, (int)few_groups_ok(r));
        for (int kv = 0; kv < 2; ++kv) {
          std::printf("%s[", kv ? ", " : "");
          for (int s = 0; s < r.rs; ++s) std::printf("%s%d", s ? ", " : "", few_raw_bar(r.rs, kv, s));
          std::printf("]");
        }
        std::printf("]}");
        sep = ", ";
      }
  std::printf("]");
}
"""

PRINT_ROWS = """
#include <cstdio>
#include "tree_rings.h"
using namespace m4q;
int main() {
  const char* sep = "[";
  for (int d = 64; d <= 128; d += 64)
    for (int q8 = 0; q8 < 2; ++q8) {
      const RowsRings r = rows_rings(d, q8 != 0);
      std::printf("%s{\\"d\\": %d, \\"q8\\": %d, \\"ks\\": %d, \\"vs\\": %d, \\"rs\\": %d, \\"sb\\": %d, \\"k_bar\\": [",
                  sep, d, q8, r.ks, r.vs, r.rs, r.sb);
      for (int t = 0; t < 2; ++t) {
        std::printf("%s[", t ? ", " : "");
        for (int s = 0; s < r.ks; ++s) std::printf("%s%d", s ? ", " : "", rows_k_bar(r.ks, t, s));
        std::printf("]");
      }
      std::printf("], \\"max_slots\\": %d, \\"max_slot\\": [", rows_max_slots(r.sb));
      for (int g = 0; g < 4; ++g) std::printf("%s%d", g ? ", " : "", rows_max_slot(r.sb, g));
      std::printf("]}");
      sep = ", ";
    }
  std::printf("]");
}
"""


def rings(tmp_path, source):
    src, exe = tmp_path / "rings.cpp", tmp_path / "rings"
    src.write_text(source)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, "-o", str(exe), str(src)], check=True)
    return json.loads(subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout)


def walk(kernel, geo, roles, seeds):
    """Every run list with every held thing; the first fault is raised."""
    for runs in RUNS:
        tiles = sum(n for n, _ in runs)
        for held in model.held_things(tiles, roles):
            for seed in range(seeds):
                kernel(geo, bool(geo["q8"]), runs, seed, held)


def test_few_rows(tmp_path):
    all_rings = rings(tmp_path, PRINT_FEW)
    assert len(all_rings) == 8
    for geo in all_rings:
        assert geo["ok"]
        walk(model.few, geo, model.FEW_ROLES, 2)


def test_the_walk_finds_a_shared_landing_barrier(tmp_path):
    # one barrier a raw slot: wrong where the ring is odd, as K and V warps then
    # wait for it in turn, and right where a slot always has one kind
    for geo in rings(tmp_path, PRINT_FEW):
        if not geo["q8"]:
            continue
        geo["raw_bar"] = [list(range(geo["rs"]))] * 2
        if geo["rs"] % 2:
            with pytest.raises(model.Fault):
                walk(model.few, geo, model.FEW_ROLES, 2)
        else:
            walk(model.few, geo, model.FEW_ROLES, 1)


def test_many_rows(tmp_path):
    all_rings = rings(tmp_path, PRINT_ROWS)
    assert len(all_rings) == 4
    for geo in all_rings:
        assert max(geo["max_slot"]) < geo["max_slots"]
        walk(model.rows, geo, model.ROWS_ROLES, 3)


def test_the_walk_finds_k_stages_shared_by_two_issuers(tmp_path):
    # one barrier a K stage: wrong with three stages and two score buffers
    for geo in rings(tmp_path, PRINT_ROWS):
        geo["k_bar"] = [list(range(geo["ks"]))] * 2
        if geo["ks"] % 2:
            assert geo["sb"] == 2
            with pytest.raises(model.Fault):
                walk(model.rows, geo, model.ROWS_ROLES, 3)
        else:
            walk(model.rows, geo, model.ROWS_ROLES, 1)


def test_the_walk_finds_one_place_for_the_maxima(tmp_path):
    # one place for the maxima of all tiles: wrong with a third score buffer, whose
    # scores do not wait for P of the last tile
    for geo in rings(tmp_path, PRINT_ROWS):
        geo["max_slot"] = [0] * 4
        if geo["sb"] == 3:
            with pytest.raises(model.Fault, match="maximum"):
                walk(model.rows, geo, model.ROWS_ROLES, 3)
        else:
            walk(model.rows, geo, model.ROWS_ROLES, 1)
