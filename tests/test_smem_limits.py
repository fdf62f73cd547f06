"""The shared memory limits of kernels (csrc/lla_smem_limits.h), compiled for the host against a stand-in of
the driver: whatever kernels share an entry, a limit never sinks."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "local_linear_attention_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <map>
#include "lla_smem_limits.h"

struct Driver {
  std::map<const void*, size_t> limit;
  int sets = 0;
  bool fail = false;
};

int main() {
  lla::SmemLimits limits;
  Driver d;
  auto ensure = [&](const void* k, size_t bytes) {
    return limits.ensure(
        k, 0, bytes, [&](size_t* held) { *held = d.limit.count(k) ? d.limit[k] : 48 * 1024; return d.fail ? 1 : 0; },
        [&](size_t most) { ++d.sets; d.limit[k] = most; return d.fail ? 2 : 0; });
  };
  const void* a = (const void*)0x1000;
  const void* b = a;  // another kernel with the same entry
  do b = (const char*)b + 16;
  while (lla::SmemLimits::slot(b, 0) != lla::SmemLimits::slot(a, 0));
  if (ensure(a, 160000) || d.limit[a] != 160000) return 1;
  if (ensure(b, 100000) || d.limit[b] != 100000) return 2;
  if (ensure(a, 60000) || d.limit[a] != 160000) return 3;  // the entry was b's: the limit stays
  if (ensure(a, 160000) || d.limit[a] != 160000) return 4;
  if (d.sets != 2) return 5;
  if (ensure(a, 170000) || d.limit[a] != 170000 || d.sets != 3) return 6;
  if (ensure(b, 1000) || d.limit[b] != 100000) return 7;
  d.fail = true;
  if (!ensure(a, 180000)) return 8;
  d.fail = false;
  if (ensure(a, 180000) || d.limit[a] != 180000) return 9;
  puts("ok");
  return 0;
}
"""


def test_limits_never_sink(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no g++")
    src = tmp_path / "limits.cc"
    src.write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-Wall", "-pthread", "-I", CSRC, str(src), "-o", str(tmp_path / "limits")], check=True)
    run = subprocess.run([str(tmp_path / "limits")], capture_output=True, text=True)
    assert (run.returncode, run.stdout) == (0, "ok\n")
