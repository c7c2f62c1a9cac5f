"""The table of shared-memory limits (csrc/smem_limit.h), compiled for the host
with a setter that only records: every kernel on every device has its own
entry, a limit is set once and never lowered."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SOURCE = r"""
#include <stdio.h>
#include <stdint.h>
#include <map>
#include <thread>
#include <utility>
#include <vector>
#include "smem_limit.h"

int main() {
  static sd::SmemLimits limits;
  std::map<std::pair<const void*, int>, size_t> now;  // written under the table's lock
  int calls = 0, lowered = 0, failed = 0;
  auto want = [&](int kern, int dev, size_t bytes) {
    const void* k = reinterpret_cast<const void*>(static_cast<uintptr_t>(kern + 1));
    const int err = limits.raise(k, dev, bytes, [&](size_t b) {
      ++calls;
      size_t& at = now[{k, dev}];
      lowered += b < at;
      at = b;
      return 0;
    });
    failed += err != 0;
  };
  const int kernels = 60, devices = 8;
  for (int pass = 0; pass < 3; ++pass)
    for (int d = 0; d < devices; ++d)
      for (int k = 0; k < kernels; ++k) want(k, d, 50000);
  printf("%d ", calls == kernels * devices);
  // threads with different sizes of the last kernels
  std::vector<std::thread> ts;
  for (int t = 0; t < 4; ++t)
    ts.emplace_back([&, t] { for (int i = 0; i < 2000; ++i) want(kernels - 1 - i % 3, i % devices, 50000 + 1000 * t); });
  for (auto& t : ts) t.join();
  int high = 0;
  for (int d = 0; d < devices; ++d)
    for (int k = kernels - 3; k < kernels; ++k) high += now[{reinterpret_cast<const void*>(static_cast<uintptr_t>(k + 1)), d}] == 53000;
  printf("%d %d %d ", lowered == 0, failed == 0, high == 3 * devices);
  // a setter's error is returned and leaves no entry behind
  int again = 0;
  const int e1 = limits.raise(&limits, 0, 1, [](size_t) { return 7; });
  const int e2 = limits.raise(&limits, 0, 1, [&](size_t) { ++again; return 0; });
  printf("%d ", e1 == 7 && e2 == 0 && again == 1);
  // a full table and an unknown device are errors, not silent sets
  int room = 0;
  for (int k = 0; k < 1000; ++k) room |= limits.raise(reinterpret_cast<const void*>(static_cast<uintptr_t>(k + 1)), 9, 1, [](size_t) { return 0; });
  printf("%d\n", room != 0 && limits.raise(&room, -1, 1, [](size_t) { return 0; }) != 0);
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_limits_are_set_once_and_never_lowered(tmp_path):
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-I", os.path.join(ROOT, "top_sparse_decode_paged_b200", "csrc"),
                    str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True, timeout=60).stdout
    assert out.split() == ["1"] * 6, out
