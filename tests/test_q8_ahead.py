"""The loads of an 8-bit attention block (csrc/q8_ahead.cuh): for shares of any length, every tile that is loaded is one that the
warp goes on to attend, in its ring place and with its own row, and every tile of codes is loaded once.

The header is compiled for the host, with arrays in the place of a warp's lanes, and driven as k_kv8_attend drives it. (A load
that no tile waits for would land in the shared memory of a block that may have ended.)"""
import os
import shutil
import subprocess

import pytest

from conftest import ROOT

SOURCE = r"""
#include <cstdio>
#include <initializer_list>
#include "q8_ahead.cuh"

struct Batch {
  int at[32];
  int row(int i) const { return at[i]; }
};

// n tiles; one of codes has a row of its own, the first `open` of every `segment` tiles have none (a segment's open blocks).
static int share(int n, int depth, int segment, int open) {
  auto want = [&](int k) { return k < n && k % segment >= open ? 1000 + k : -1; };
  auto look_up = [&](int k0) {
    Batch b;
    for (int i = 0; i < 32; ++i) b.at[i] = want(k0 + i);
    return b;
  };
  Batch none;
  for (int i = 0; i < 32; ++i) none.at[i] = -1;
  lfm3::Q8Ahead<Batch> ahead{look_up(0), none};
  int held[8];  // the row that is on its way to, or lies in, a place of the ring
  for (int p = 0; p < depth; ++p) held[p] = ahead.row(p, 0);
  for (int k = 0; k < n; ++k) {
    if (held[k % depth] != want(k)) return printf("n %d depth %d segment %d open %d: tile %d has row %d, not %d\n", n, depth, segment, open, k, held[k % depth], want(k)), 1;
    if (ahead.cur.at[k & 31] != want(k)) return printf("n %d: the batch of tile %d is another one's\n", n, k), 1;
    held[k % depth] = ahead.row(k + depth, k);
    ahead.done(k, look_up);
  }
  for (int p = 0; p < depth; ++p)
    if (held[p] != -1) return printf("n %d depth %d segment %d open %d: row %d is loaded and never attended\n", n, depth, segment, open, held[p]), 1;
  return 0;
}

int main() {
  for (int n = 1; n <= 400; ++n)
    for (int depth = 2; depth <= 4; ++depth)
      for (int segment : {1000, 97, 40, 31, 5})
        for (int open : {0, 1, 2})
          if (share(n, depth, segment, open)) return 1;
  return 0;
}
"""


def test_every_load_is_attended(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no g++")
    src, exe = tmp_path / "ahead.cpp", tmp_path / "ahead"
    src.write_text(SOURCE)
    csrc = os.path.join(ROOT, "attention_decoder_b200", "csrc")
    subprocess.run([cxx, "-std=c++17", "-O1", "-I", csrc, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
