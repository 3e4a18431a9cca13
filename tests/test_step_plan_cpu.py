"""The arithmetic of a step's plan, compiled for the host from the kernels' own header: the parts that a job is cut
into.  A sequence's partial rows lie `parts of its last row tile` apart, so no earlier row tile, which has fewer keys,
may have more parts: its rows would be another tile's."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "transformer_sharding_affinity_gb300", "csrc")
CUDA = os.environ.get("CUDA_HOME", "/usr/local/cuda")

# the device functions of step.cuh as plain ones
PROGRAM = r"""
#include <cuda_runtime.h>
#include <algorithm>
#include <cstdio>
using std::min;
using std::max;
#define __CUDACC__ 1
#undef __device__
#undef __host__
#undef __forceinline__
#define __device__
#define __host__
#define __forceinline__ inline
#include "step.cuh"

int main() {
  for (int streams = 1; streams <= 2; ++streams)
    for (int unit = 0; unit <= 300; ++unit) {
      int before = 0;
      for (int tiles = 0; tiles <= 700; ++tiles) {
        int per = -1;
        const int parts = aff::job_parts(tiles, streams, unit, &per);
        const bool covers = tiles == 0 ? parts == 1 && per == 0
                                       : parts >= 1 && per >= 1 && parts * per >= tiles && (parts - 1) * per < tiles;
        const bool within = unit == 0 ? parts == 1 : per * streams <= unit + streams - 1;
        if (!covers || !within || parts < before) {
          std::printf("streams %d unit %d tiles %d: %d parts of %d, %d before\n", streams, unit, tiles, parts, per, before);
          return 1;
        }
        before = parts;
      }
    }
  return 0;
}
"""


def test_a_job_with_more_keys_has_no_fewer_parts(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None or not os.path.exists(os.path.join(CUDA, "include", "cuda_runtime.h")):
        pytest.skip("needs a C++ compiler and the CUDA headers")
    (tmp_path / "parts.cpp").write_text(PROGRAM)
    exe = str(tmp_path / "parts")
    subprocess.run([gxx, "-O1", "-w", "-std=c++17", "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-I",
                    os.path.join(CUDA, "include"), str(tmp_path / "parts.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], stdout=subprocess.PIPE, text=True)
    assert r.returncode == 0, r.stdout
