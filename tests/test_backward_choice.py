"""The shaped backward's choice between shares per query head and groups in one item, on the host alone."""
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
  const int shape[][5] = {{1, 8, 2, 997, 64}, {1, 32, 8, 2048, 128}, {1, 32, 8, 4096, 128}, {1, 8, 8, 997, 64}};
  for (auto& s : shape) {
    fattn::BwdParams p{};
    p.B = s[0]; p.Hq = s[1]; p.Hkv = s[2]; p.N = s[3]; p.d = s[4]; p.causal = 1;
    printf("%d%d%d ", fattn::bwd_per_head(p, 152), fattn::bwd_per_head(p, 76), fattn::bwd_per_head(p, 4));
  }
}
"""


def test_choice_follows_the_sms(tmp_path):
    """Few items of few heads on many SMs take the heads apart; on four SMs, which the items fill, nothing is won by it."""
    cuda = "/usr/local/cuda/include"
    if not (shutil.which("g++") and os.path.isdir(cuda)):
        pytest.skip("needs g++ and the CUDA headers")
    src, exe = tmp_path / "choice.cpp", tmp_path / "choice"
    src.write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-I" + CSRC, "-I" + os.path.join(ROOT, "include"), "-I" + cuda, str(src), "-o", str(exe)],
                   check=True)
    got = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()
    assert got == ["110", "100", "000", "000"]
