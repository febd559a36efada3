"""The streaming kernel's choice between clusters and the line of steps, on the host alone."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "exact_tiled_attention_fattn_gb300", "csrc")
SOURCE = """
#include "ops_internal.h"
#include <cstdio>
int main() {
  fattn::StreamFp8Params p{};
  p.subs = 1; p.page_size = 16; p.max_q = 1; p.causal = 1; p.B = 1; p.Hkv = 4; p.num_splits = 77;
  p.max_pages = 30000 / 16;
  for (int most : {16, 8, 4, 2, 1}) printf("%d ", fattn::stream_fp8_cluster(p, 12, 152, most));
  p.max_pages = 2000 / 16;
  for (int most : {16, 8, 4, 2, 1}) printf("%d ", fattn::stream_fp8_cluster(p, 12, 152, most));
  p.num_splits = 5;
  printf("%d ", fattn::stream_fp8_cluster(p, 12, 152, 16));
  p.num_splits = 1;
  printf("%d | ", fattn::stream_fp8_cluster(p, 12, 152, 16));
  // 152 groups beside a window: with causal a step or two of work, else as much again behind the queries
  p.num_splits = 9; p.B = 19; p.Hkv = 8; p.max_pages = 4000;
  for (int window : {100, 200, 400, 800, 1600})
    for (int causal : {1, 0}) {
      p.causal = causal; p.shape.window = window;
      const int both = fattn::stream_fp8_cluster(p, 12, 152, 16);
      p.causal = 1; p.shape.window = causal ? window : 2 * window;
      printf("%d ", both == fattn::stream_fp8_cluster(p, 12, 152, 16));
    }
}
"""


def test_clusters(tmp_path):
    """No more CTAs than the device has room for, nor than the pieces that the caller allows; 30000 tokens of one context go
    to the line where clusters of 16 find no room; of 2000 (125 steps) two CTAs take 6 + 3, the line 1 + 8 + 1. A window without causal counts on both sides."""
    cuda = "/usr/local/cuda/include"
    if not (shutil.which("g++") and os.path.isdir(cuda)):
        pytest.skip("needs g++ and the CUDA headers")
    src, exe = tmp_path / "clusters.cpp", tmp_path / "clusters"
    src.write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-I" + CSRC, "-I" + os.path.join(ROOT, "include"), "-I" + cuda, str(src), "-o", str(exe)],
                   check=True)
    got = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout
    assert got == "16 0 0 0 0 16 8 4 2 0 4 1 | 1 1 1 1 1 1 1 1 1 1 ", got
