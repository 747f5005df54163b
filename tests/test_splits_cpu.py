"""The rules by which a cross attention's states are shared out over the blocks of a cluster (host code, no GPU):
the header is compiled by the host compiler and asked over a range of sizes."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "speech_recognition_audio_b200", "csrc")

PROGRAM = r"""
#include <cstdio>
#include "splits.h"
int main() {
  int asked = 0;
  for (int s = 1; s <= 16; s *= 2) {
    // a device that cannot hold 16 blocks gets 8, and is only asked where it matters
    if (asr::cap_splits(s, [&] { ++asked; return false; }) != (s > 8 ? 8 : s)) return 1;
    if (asr::cap_splits(s, [&] { ++asked; return true; }) != s) return 2;
  }
  if (asked != 2) return 3;
  for (long long blocks = 1; blocks < 5000; blocks = blocks * 3 / 2 + 1)
    for (int keys = 0; keys < 40000; keys = keys * 2 + 1)
      for (int most = 8; most <= 16; most *= 2) {
        const int s = asr::pick_splits(blocks, keys, 64, 1480, most);
        if (s < 1 || s > most || (s & (s - 1))) return 4;
        if (s > 1 && (keys < s * 64 || blocks * (s / 2) >= 1480)) return 5;
        const int t = asr::tile_splits((double)blocks, (keys + 127) / 128, 12.5, 148);
        if (t < 1 || t > 16 || (t & (t - 1))) return 6;
        if (t > 1 && (t > (keys + 127) / 128 || blocks * t > 2 * 148)) return 7;
      }
  puts("ok");
  return 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="no host compiler")
def test_split_rules(tmp_path):
    src, exe = tmp_path / "splits.cpp", tmp_path / "splits"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-I", CSRC, str(src), "-o", str(exe)], check=True, timeout=120)
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert run.returncode == 0 and run.stdout == "ok\n", run.returncode
