"""CPU test of the main matrix product's load addresses: csrc/load_bounds.h, the code the kernel
computes them with, replayed by a host program over short sums, ragged outer sizes and padded rows.
Every 16-byte load that its buffer resource lets through lies inside the operand's array, and every
value of the operand is loaded."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "mxfp8_block_scaled_partial_amd", "csrc")

PROGRAM = r"""
#include <stdio.h>
#include <stdlib.h>

#include <vector>

#include "load_bounds.h"

using namespace mxfp8;

static long loads = 0;

// Array [rows][ld], `width` bytes of each row in use: (rows, width) = (outer, k) or (k, outer).
template <int T, bool kRows>
static void replay(int64_t outer, int64_t k, int64_t ld) {
  const int64_t rows = kRows ? k : outer, width = kRows ? outer : k;
  const int64_t bytes = (rows - 1) * ld + width;
  std::vector<char> seen(rows * ld, 0);
  for (int64_t outer0 = 0; outer0 < outer; outer0 += T) {
    const int halves = (int)((2 * ((k + 127) / 128) + 3) & ~3);
    for (int half = 0; half < halves; ++half) {
      const int64_t k0 = int64_t(half) * kHalf;
      const int left = (int)(k - k0);
      const int64_t base = kRows ? k0 * ld + outer0 : outer0 * ld + k0;
      const uint32_t extent = kRows ? rows_extent(left, (int)ld, outer - outer0) : cols_extent<T>(outer - outer0, ld);
      for (int slot = 0; slot < T * kHalf / 16; ++slot) {
        const Place p = place_of<T, kRows>(slot);
        uint32_t off = (uint32_t)(p.row * (int)ld + p.at);
        if (!kRows) off = cols_offset(off, p.at, left);
        for (int i = 0; i < 16; ++i) {  // the resource checks each dword; this checks each byte
          if (uint64_t(off) + i >= extent) continue;
          const int64_t at = base + off + i;
          ++loads;
          if (at < 0 || at >= bytes) {
            printf("T=%d %s outer=%ld k=%ld ld=%ld: byte %ld of %ld\n", T, kRows ? "rows" : "cols", (long)outer, (long)k,
                   (long)ld, (long)at, (long)bytes);
            exit(1);
          }
          seen[at] = 1;
        }
      }
    }
  }
  for (int64_t r = 0; r < rows; ++r)
    for (int64_t c = 0; c < width; ++c)
      if (!seen[r * ld + c]) {
        printf("T=%d %s outer=%ld k=%ld ld=%ld: row %ld byte %ld is not loaded\n", T, kRows ? "rows" : "cols", (long)outer,
               (long)k, (long)ld, (long)r, (long)c);
        exit(1);
      }
}

template <int T>
static void tile() {
  const int64_t outers[] = {1, 15, 16, 17, 32, 48, 63, 64, 100, 128, 144, 192, 208, 255, 256, 257, 300, 320};
  const int64_t sums[] = {16, 32, 48, 64, 80, 112, 128, 144, 256, 272, 528};
  const int64_t pads[] = {0, 16, 48, 64, 1024};
  for (int64_t outer : outers)
    for (int64_t k : sums)
      for (int64_t pad : pads) {
        replay<T, false>(outer, k, k + pad);
        if (outer % 16 == 0) {
          replay<T, true>(outer, k, outer + pad);
          replay<T, true>(outer, k - 15, outer + pad);
        }
      }
}

int main() {
  tile<256>();
  tile<192>();
  tile<128>();
  tile<64>();
  printf("%ld loads inside\n", loads);
  return 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs the host C++ compiler")
def test_every_load_is_inside_its_operand(tmp_path):
    src, exe = tmp_path / "replay.cpp", tmp_path / "replay"
    src.write_text(PROGRAM)
    subprocess.check_call(["g++", "-std=c++17", "-O2", "-Wall", "-Werror", f"-I{CSRC}", str(src), "-o", str(exe)])
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout
    assert "loads inside" in r.stdout
