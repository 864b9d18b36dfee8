"""Where the codes of an FP8_BLOCK block lie: the header's own functions, compiled for the
host, against the order that its text states.  (That the kernels seal and read by it is
what the GPU tests of sealed bytes and of decode show.)"""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "decode_attention_pruned_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#define __host__
#define __device__
#define __forceinline__ inline
#include "lk_block.h"
int main() {
  for (int k = 32; k <= 128; k += 32) {
    std::printf("size %d %d %d %d\n", k, lk::block_voff(k), lk::block_soff(k), lk::block_bytes(k));
    for (int r = 0; r < 128; ++r)
      for (int c = 0; c < k; ++c) std::printf("k %d %d %d %d\n", k, r, c, lk::block_kbyte(k, r, c));
  }
  for (int r = 0; r < 128; ++r)
    for (int c = 0; c < 128; ++c) std::printf("v 0 %d %d %d\n", r, c, lk::block_vbyte(r, c));
}
"""


def _stated():
    """{(what, k, row, channel): byte}: K word of lane 4 g + t of slab s and unit u at 16 k s + 512 u +
    16 lane, channels 32 u + 8 t + 0 .. 7 of row 16 s + g, then of row 16 s + g + 8; V word of
    lane 4 g + t and unit u at 2048 s + 512 u + 16 lane: for channel 8 g + 2 u, its 64th
    successor, channel 8 g + 2 u + 1, its 64th successor: rows 16 s + 2 t, 2 t + 1, 2 t + 8, 2 t + 9."""
    at = {}
    for s in range(8):
        for g in range(8):
            for t in range(4):
                lane = 4 * g + t
                for k in (32, 64, 96, 128):
                    for u in range(k // 32):
                        word = 16 * k * s + 512 * u + 16 * lane
                        for j in range(16):
                            at["k", k, 16 * s + g + 8 * (j // 8), 32 * u + 8 * t + j % 8] = word + j
                for u in range(4):
                    word = 2048 * s + 512 * u + 16 * lane
                    channels = [8 * g + 2 * u, 64 + 8 * g + 2 * u, 8 * g + 2 * u + 1, 64 + 8 * g + 2 * u + 1]
                    rows = [16 * s + 2 * t, 16 * s + 2 * t + 1, 16 * s + 2 * t + 8, 16 * s + 2 * t + 9]
                    for j in range(16):
                        at["v", 0, rows[j % 4], channels[j // 4]] = word + j
    return at


def _compiled(tmp_path, header_dir):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no host C++ compiler")
    src, exe = tmp_path / "layout.cc", tmp_path / "layout"
    src.write_text(PROGRAM)
    subprocess.run([gxx, "-std=c++17", "-I", header_dir, "-I", CSRC, "-I", os.path.join(ROOT, "include"), str(src),
                    "-o", str(exe)], check=True)
    sizes, at = {}, {}
    for line in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines():
        what, *x = line.split()
        x = [int(y) for y in x]
        if what == "size":
            sizes[x[0]] = tuple(x[1:])
        else:
            at[what, x[0], x[1], x[2]] = x[3]
    return sizes, at


def test_header_lays_codes_as_it_says(tmp_path):
    sizes, at = _compiled(tmp_path, CSRC)
    assert at == _stated()
    assert sizes == {k: (128 * k, 128 * (k + 128), 128 * (k + 128) + 16) for k in (32, 64, 96, 128)}


@pytest.mark.parametrize("good, bad", [("((r >> 3) & 1) * 8 + (c & 7)", "((r >> 3) & 1) * 8 + (c & 3)"),
                                       ("((r >> 3) & 1) * 2 + (r & 1)", "((r >> 3) & 1) + (r & 1) * 2")])
def test_a_header_with_another_order_is_found_out(tmp_path, good, bad):
    """A copy of the header that places some codes elsewhere."""
    text = open(os.path.join(CSRC, "lk_block.h")).read()
    assert text.count(good) == 1
    (tmp_path / "lk_block.h").write_text(text.replace(good, bad))
    assert _compiled(tmp_path, str(tmp_path))[1] != _stated()
