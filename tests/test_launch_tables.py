"""csrc/launch_tables.h under several threads, with fakes of the driver's calls."""
import os
import subprocess

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "mxfp4_routed_expert_moe_gb300", "csrc")
PROGRAM = r"""
#include "launch_tables.h"
#include <atomic>
#include <chrono>
#include <cstdio>
#include <thread>
#include <vector>

static void nap(int us) { std::this_thread::sleep_for(std::chrono::microseconds(us)); }

int main() {
  static int kernels[40];
  // Two threads ask for a large and for a small size at the same time: what is set at the end serves both.
  for (int k = 0; k < 40; ++k) {
    static moe::SmemTable table;
    std::atomic<size_t> set{0};
    std::atomic<int> calls{0};
    auto ask = [&](size_t bytes, int wait) {
      return table.ensure(&kernels[k], bytes, [&](const void*, size_t n) {
        ++calls;
        nap(wait);
        set = n;
        return 0;
      });
    };
    std::thread a([&] { ask(100000, k % 2 ? 100 : 2000); }), b([&] { ask(50000, k % 2 ? 2000 : 100); });
    a.join();
    b.join();
    if (set < 100000) return std::printf("kernel %d is left with %zu bytes\n", k, set.load()), 1;
    const int before = calls;
    if (ask(100000, 0) || ask(70000, 0) || calls != before) return std::printf("asked again\n"), 1;
    if (ask(100001, 0) || calls != before + 1 || set != 100001) return std::printf("not raised\n"), 1;
  }
  // A refusal is returned and not kept.
  moe::SmemTable table;
  if (table.ensure(&kernels[0], 9, [](const void*, size_t) { return 3; }) != 3) return 2;
  if (table.ensure(&kernels[0], 9, [](const void*, size_t) { return 4; }) != 4) return 2;
  if (table.ensure(&kernels[0], 9, [](const void*, size_t) { return 0; }) != 0) return 2;
  if (table.ensure(&kernels[0], 8, [](const void*, size_t) { return 5; }) != 0) return 2;
  // Occupancies: every thread reads what belongs to its question.
  static moe::OccupancyTable occ;
  std::atomic<int> wrong{0};
  std::vector<std::thread> threads;
  for (int t = 0; t < 8; ++t)
    threads.emplace_back([&, t] {
      for (int i = 0; i < 500; ++i) {
        const int k = (i * 7 + t) % 40;
        int ctas = -1;
        if (occ.get(&kernels[k], 32 * (1 + k % 3), 100 + k, &ctas, [&](const void*, int n, size_t, int* out) {
              nap(20);
              *out = n + k;
              return 0;
            }) || ctas != 32 * (1 + k % 3) + k)
          ++wrong;
      }
    });
  for (auto& t : threads) t.join();
  int ctas = -1;
  if (occ.get(&kernels[0], 7, 7, &ctas, [](const void*, int, size_t, int*) { return 6; }) != 6 || ctas != -1) return 3;
  if (occ.get(&kernels[0], 7, 7, &ctas, [](const void*, int, size_t, int* out) { return *out = 0; }) != 0 || ctas != 1) return 3;
  return wrong ? 4 : 0;
}
"""


@pytest.mark.parametrize("flags", [["-O2"], ["-O1", "-g"]])
def test_tables_under_threads(tmp_path, flags):
    src, exe = tmp_path / "tables.cpp", tmp_path / "tables"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", *flags, "-I", CSRC, str(src), "-o", str(exe), "-pthread"], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout
