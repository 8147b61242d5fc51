"""First calls from many threads at once: what the library finds out about a device once
(csrc/per_device.h) is found out by one of them, and never written after another may
read it (no GPU needed)."""
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "swiglu_block_quantized_gb300", "csrc")

THREADS = r"""
#include <atomic>
#include <chrono>
#include <cstdio>
#include <thread>
#include <vector>
#include "per_device.h"
struct Facts { int a = 0, b = 0; };
int main() {
  static m4q::PerDevice<Facts, 4> all;
  static std::atomic<int> made[4], wrong, go, fail{FAILS};
  std::vector<std::thread> t;
  for (int i = 0; i < 32; ++i)
    t.emplace_back([i] {
      const int id = i % 4;
      while (!go.load()) {}
      Facts f;
      for (;;) {
        const int rc = all.get(id, &f, [id](Facts* k) {
          if (fail.fetch_sub(1) > 0) return -5;
          k->a = id + 1;
          std::this_thread::sleep_for(std::chrono::milliseconds(30));   // the others arrive meanwhile
          k->b = 10 * (id + 1);
          ++made[id];
          return 0;
        });
        if (rc == 0) break;
        if (rc != -5) ++wrong;
      }
      if (f.a != id + 1 || f.b != 10 * (id + 1)) ++wrong;
    });
  go = 1;
  for (auto& x : t) x.join();
  std::printf("%d %d %d %d %d", made[0].load(), made[1].load(), made[2].load(), made[3].load(), wrong.load());
}
"""


@pytest.mark.parametrize("fails", [0, 3])
def test_one_thread_finds_out(tmp_path, fails):
    src, exe = tmp_path / "threads.cpp", tmp_path / "threads"
    src.write_text(THREADS.replace("FAILS", str(fails)))
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-pthread", "-I", CSRC, "-o", str(exe), str(src)],
                   check=True)
    assert subprocess.run([str(exe)], check=True, capture_output=True, text=True, timeout=60).stdout == "1 1 1 1 0"


def test_the_library_asks_through_it():
    with open(os.path.join(CSRC, "api.cu")) as f:
        code = f.read()
    body = code[code.index("int ready(DevInfo* dev"):code.index("int done(cudaError_t e)")]
    assert "PerDevice<" in body and "known" not in body
