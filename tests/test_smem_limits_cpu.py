"""The record of the kernels' shared-memory limits: any number of kernels and devices, limits that only grow."""
import os
import subprocess

from doge_dynamic_mask_b200 import build

PROGRAM = r"""
#include <atomic>
#include <cstdio>
#include <thread>
#include <vector>
#include "smem_limits.h"

std::atomic<int> limit_of[400][2];   // what the runtime would hold (set() runs under the record's lock)
int lowered, calls;

int main() {
  static dma::SmemLimits limits;
  auto ask = [&](int f, int dev, int bytes) {
    return limits.raise(&limit_of[f], dev, bytes, [&] {
      ++calls;
      if (bytes > 232448) return 1;
      if (bytes < limit_of[f][dev]) ++lowered;
      limit_of[f][dev] = bytes;
      return 0;
    });
  };
  for (int f = 0; f < 400; ++f)   // every kernel on both devices, a large launch and then a small one
    for (int dev = 0; dev < 2; ++dev)
      if (ask(f, dev, 100000 + f) || ask(f, dev, 50000)) return 1;
  const int first = calls;
  for (int f = 0; f < 400; ++f)
    if (ask(f, 1, 100000 + f)) return 2;
  const int again = calls - first;
  if (ask(7, 0, 300000) != 1 || ask(7, 0, 100007) != 0) return 3;   // a refusal grants nothing and takes nothing away
  // a large launch that finds less than it was promised, while another thread prepares small ones
  std::atomic<int> short_of{0};
  std::vector<std::thread> threads;
  for (int t = 0; t < 4; ++t)
    threads.emplace_back([&, t] {
      for (int i = 0; i < 20000; ++i) {
        const int f = i % 400, bytes = t % 2 ? 60000 : 200000 + f;
        ask(f, 0, bytes);
        if (limit_of[f][0] < bytes) ++short_of;
      }
    });
  for (auto& t : threads) t.join();
  std::printf("%d %d %d %d\n", first, again, lowered, short_of.load());
  return 0;
}
"""


def test_any_number_of_kernels_and_no_limit_lowered(tmp_path):
    (tmp_path / "p.cpp").write_text(PROGRAM)
    exe = str(tmp_path / "p")
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-I" + build.CSRC, str(tmp_path / "p.cpp"), "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert out.returncode == 0
    first, again, lowered, short = map(int, out.stdout.split())
    assert first == 800        # one grant per kernel and device: the small launches needed none
    assert (again, lowered, short) == (0, 0, 0)
