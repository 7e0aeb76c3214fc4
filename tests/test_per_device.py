"""The cache of what a device is asked once: an answer per device, failures reported and not kept.  The
header is compiled with the host compiler into a small program (CPU)."""

import os
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "memory_bounded_linear_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <thread>
#include <vector>
#include "per_device.h"
enum Error { ok = 0, bad = 7 };
lce::PerDevice<4> cache;
int main() {
  int asked = 0, v = -1;
  auto says = [&](int n) { return [&asked, n](int* out) { ++asked; *out = n; return ok; }; };
  auto fails = [&](int* out) { ++asked; *out = 99; return bad; };
  if (cache.get(1, fails, &v) != bad || cache.get(1, fails, &v) != bad || asked != 2) return 1;  // not kept
  if (cache.get(1, says(38), &v) != ok || v != 38 || asked != 3) return 2;
  if (cache.get(1, fails, &v) != ok || v != 38 || asked != 3) return 3;                          // kept
  if (cache.get(3, says(0), &v) != ok || v != 0 || asked != 4) return 4;       // another device; 0 is an answer
  if (cache.get(3, says(5), &v) != ok || v != 0 || asked != 4) return 5;
  lce::PerDevice<2> shared;
  std::vector<std::thread> threads;
  std::atomic<int> wrong{0};
  for (int t = 0; t < 8; ++t)
    threads.emplace_back([&] {
      for (int i = 0; i < 2000; ++i) {
        int x = -1;
        if (shared.get(i & 1, [&](int* out) { *out = 10 + (i & 1); return ok; }, &x) != ok || x != 10 + (i & 1)) ++wrong;
      }
    });
  for (auto& t : threads) t.join();
  return wrong ? 6 : 0;
}
"""


def test_cache(tmp_path):
    src, exe = tmp_path / "p.cpp", tmp_path / "p"
    src.write_text(PROGRAM)
    subprocess.run([os.environ.get("CXX", "g++"), "-std=c++17", "-O1", "-Wall", "-pthread", f"-I{CSRC}", str(src), "-o",
                    str(exe)], check=True)
    assert subprocess.run([str(exe)]).returncode == 0


def test_feed_forward_kernels_keep_no_other_state():
    """Static variables of the launch code: the cache, nothing without a device or without atomics."""
    for name in ("lce_ffn_tc.cu", "lce_ffn_few.cu", "lce_ffn_simt.cu", "lce_ffn_api.cu", "lce_gradnorm.cu"):
        for line in open(os.path.join(CSRC, name)):
            words = line.strip().split()
            if words[:1] == ["static"] and "constexpr" not in words:
                assert words[1].startswith("PerDevice<kMaxDevices>"), (name, line)
