"""The host's queries of resident clusters where they fail (a cluster size and a device that do not
exist): no answer, and no error left behind for the next launch to report as its own."""

import os
import subprocess

import pytest

from paged_latent_attention_mla_gb300 import build as nbuild

pytestmark = pytest.mark.gpu

PROGRAM = r"""
#include <cuda_runtime_api.h>
#include <cstdio>
namespace mla {
struct ShortShape { int rows, ctas; };
int short_max_clusters(ShortShape s, bool e4m3);
int split_kv_max_clusters(int device, bool e4m3);
}
int main() {
  int bad = 0;
  auto look = [&](const char* what, int n, bool some) {
    const cudaError_t e = cudaGetLastError();
    if ((n > 0) == some && e == cudaSuccess) return;
    std::printf("%s: %d clusters, %s\n", what, n, cudaGetErrorName(e));
    bad = 1;
  };
  for (int e4m3 = 0; e4m3 < 2; ++e4m3) {
    for (int rows = 16; rows <= 64; rows *= 2) {
      look("short, 16 CTAs", mla::short_max_clusters({rows, 16}, e4m3 != 0), true);
      look("short, 32 CTAs", mla::short_max_clusters({rows, 32}, e4m3 != 0), false);
    }
    look("split", mla::split_kv_max_clusters(0, e4m3 != 0), true);
    look("split, no such device", mla::split_kv_max_clusters(9999, e4m3 != 0), false);
  }
  return bad;
}
"""


def test_failed_queries_leave_no_error(tmp_path):
    nbuild.build()
    src, exe = tmp_path / "query.cpp", tmp_path / "query"
    src.write_text(PROGRAM)
    objs = [os.path.join(nbuild.BUILD, f) for f in ("mla_short.o", "mla_split_tc.o")]
    r = subprocess.run([nbuild._nvcc(), "-arch=sm_103a", "-std=c++17", "-cudart", "static", str(src), "-o", str(exe)] + objs,
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
