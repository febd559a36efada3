"""The shaped backward's choice between query heads and groups with windows and sinks, on the host alone: the sinks' tiles are
seen from all queries, and how far they are cut decides how long the longest item is."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "exact_tiled_attention_fattn_gb300", "csrc")
SOURCE = """
#include "fattn_internal.h"
#include <cstdio>
int main() {
  // B, Hq, Hkv, N, window, sinks
  const int shape[][6] = {{1, 8, 2, 9000, 128, 4200}, {1, 8, 2, 9000, 128, 0}, {1, 8, 2, 9000, 128, 4},
                          {1, 32, 1, 16384, 128, 8000}, {1, 8, 2, 997, 100, 17}};
  for (auto& s : shape) {
    fattn::BwdParams p{};
    p.B = s[0]; p.Hq = s[1]; p.Hkv = s[2]; p.N = s[3]; p.d = 128; p.causal = 1;
    p.shape.window = s[4]; p.shape.sinks = s[5];
    p.sink_tiles = fattn::sink_blocks(s[5], 128);
    p.sink_pieces = fattn::bwd_sink_pieces(s[3], 1, s[4], s[5]);
    printf("%d/%d ", fattn::bwd_per_head(p, 152), p.sink_pieces);
  }
}
"""


def test_choice_follows_the_longest_piece(tmp_path):
    """In steps of one query tile, 152 SMs, G heads a group, items of nt / pieces steps, what joins the heads 2 + 2.6e-6 B N Hq d:
    one KV head of 32, 128 query tiles, 63 tiles of sinks in 2 pieces: groups 32 * 64 = 2048 at least, heads the SMs' mean,
    (128 * 2 + 63 * 96.5) * 32 / 152 = 1334, and 176 more: the heads apart (without the sinks' share 64 against 230). Two
    KV heads of 4, 71 query tiles, 33 tiles of sinks in 3 pieces: groups 4 * 23.7 or the mean, 102; heads 102 + 26."""
    cuda = "/usr/local/cuda/include"
    if not (shutil.which("g++") and os.path.isdir(cuda)):
        pytest.skip("needs g++ and the CUDA headers")
    src, exe = tmp_path / "choice.cpp", tmp_path / "choice"
    src.write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-I" + CSRC, "-I" + os.path.join(ROOT, "include"), "-I" + cuda, str(src), "-o", str(exe)],
                   check=True)
    got = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()
    assert got == ["0/3", "0/1", "0/24", "1/2", "1/4"], got
