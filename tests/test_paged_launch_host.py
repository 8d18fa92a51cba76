"""What the launches ask of the device, against a fake of the CUDA runtime's answers
(a host program of the launch header and the fakes).  No GPU needed."""
import os
import shutil
import subprocess

import pytest

from tile_level_overlap_gb300 import build

PROGRAM = r"""
#include <stdio.h>
#include "mk_paged.h"

static int asked = 0, fails = 0;  // which of the next answers is an error: 1 the attributes, 2 the number
extern "C" {
cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int) { return fails == 1 ? cudaErrorMemoryAllocation : cudaSuccess; }
cudaError_t cudaOccupancyMaxActiveClusters(int* n, const void*, const cudaLaunchConfig_t* c) {
  ++asked;
  *n = fails == 2 ? 99 : (int)(152 / c->gridDim.x);
  return fails == 2 ? cudaErrorMemoryAllocation : cudaSuccess;
}
cudaError_t cudaGetLastError() { return cudaSuccess; }
}

int main() {
  static std::atomic<int> known[64][17];
  auto ask = [&](int device, int ctas) { return mk::paged_clusters_at_once(&asked, 256, 1024, device, ctas, known); };
  for (int device : {0, 63, 64}) {
    for (int kind : {1, 2}) {
      const int ctas = kind == 1 ? 16 : 4;
      fails = kind;
      const int failed = ask(device, ctas);
      fails = 0;
      asked = 0;
      const int first = ask(device, ctas), again = ask(device, ctas);
      printf("%d %d %d %d\n", failed, first, again, asked);
    }
  }
  return 0;
}
"""


def test_a_failed_question_is_asked_again(tmp_path):
    cxx = shutil.which("g++") or pytest.skip("no host compiler")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build.nvcc()))), "include")
    src = tmp_path / "fake.cpp"
    src.write_text(PROGRAM)
    exe = tmp_path / "fake"
    r = subprocess.run([cxx, "-std=c++17", "-I", cuda, "-I", build.CSRC, str(src), "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert out.returncode == 0
    rows = [tuple(map(int, line.split())) for line in out.stdout.splitlines()]
    # what failed counts as none, once; the answer is then kept (devices past 63 are asked each time)
    assert rows == [(0, 9, 9, 1), (0, 38, 38, 1)] * 2 + [(0, 9, 9, 2), (0, 38, 38, 2)]
