"""The plan of the shared-prefix decode, run on the CPU from the header the kernels
include: every block of every tile lies in exactly one segment, every segment has a
slot of its own inside the workspace, and a tile's table entry names exactly the
slots of its segments."""
import ctypes
import os
import random
import subprocess

import numpy as np
import pytest

from mla_latent_kv_yarn_b200 import build as xbuild

BLOCK, ROWS, OWN_Q, HEADS, PAGE = 256, 128, 4, 32, 64

DRIVER = r"""
#include "shared_plan.h"
using namespace xmla;
// Walks every run; fills tab (first slot, count of each tile) and segs (run, own, tile,
// first block, blocks, slot, first row, sequence, tokens).  Returns the segments, or -1.
extern "C" int walk(int batch, int q_len, int prefix_pages, long long max_seqlen, const int* lens,
                    int tiles, int blocks, int own_tiles, int pairs, int* tab, long long* segs, int most) {
  SharedParams p{};
  p.seqlens = lens;
  p.batch = batch; p.q_len = q_len; p.prefix_pages = prefix_pages; p.max_seqlen = max_seqlen;
  p.tiles = tiles; p.blocks = blocks; p.own_tiles = own_tiles; p.pairs = pairs;
  int* cum = new int[batch + 1];
  cum[0] = 0;
  for (int b = 0; b < batch; ++b) cum[b + 1] = cum[b] + (own_tiles ? own_places(p, b) : 0);
  const SharedWork w = shared_work(p, cum[batch]);
  for (int t = 0; t < tiles + batch * own_tiles; ++t) {
    const int2 v = shared_tile_partials(p, w, t, cum);
    tab[2 * t] = v.x;
    tab[2 * t + 1] = v.y;
  }
  int n = 0;
  for (int run = 0; run < pairs; ++run) {
    Segments s{};
    s.at = shared_run(p, w, run, cum);
    while (s.next(p)) {
      if (n == most) return -1;
      const long long v[9] = {run, s.is_own, s.tile, s.b0, s.n, s.slot(run), s.row0(p), s.is_own ? s.seq : -1,
                              s.is_own ? s.tokens : -1};
      for (int k = 0; k < 9; ++k) segs[9 * n + k] = v[k];
      ++n;
    }
  }
  delete[] cum;
  return n;
}
"""


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    src, lib = d / "plan.cu", d / "plan.so"
    src.write_text(DRIVER)
    subprocess.run([xbuild._nvcc(), "-gencode", "arch=compute_100a,code=sm_100a", "-O1", "-std=c++17", "-Xcompiler",
                    "-fPIC", "-shared", "-I", xbuild.CSRC, str(src), "-o", str(lib)], check=True)
    f = ctypes.CDLL(str(lib)).walk
    ll = ctypes.c_longlong
    f.argtypes = [ctypes.c_int] * 3 + [ll, ctypes.c_void_p] + [ctypes.c_int] * 4 + [ctypes.c_void_p] * 2 + [ctypes.c_int]
    return f


def check(walk, batch, q_len, pages, own, room, copied, sms):
    lens = np.array([pages * PAGE + n for n in own], dtype=np.int32)
    longest = pages * PAGE + room
    tiles, blocks = -(-batch * q_len * HEADS // ROWS), -(-pages * PAGE // BLOCK)
    own_tiles = -(-q_len // OWN_Q) if copied else 0
    places = tiles * (blocks + 1) + batch * own_tiles * (-(-room // BLOCK) + 1)
    pairs = min(sms // 2, 128, places)
    tab = np.full((tiles + batch * own_tiles, 2), -1, dtype=np.int32)
    segs = np.zeros((pairs + tiles + batch * own_tiles, 9), dtype=np.int64)
    n = walk(batch, q_len, pages, longest, lens.ctypes.data, tiles, blocks, own_tiles, pairs, tab.ctypes.data,
             segs.ctypes.data, len(segs))
    assert n >= 0, "more segments than tiles and runs"
    good = [o if q_len <= o <= room else 0 for o in own]
    want = {(0, t): blocks for t in range(tiles)}
    for t in range(batch * own_tiles):
        want[1, t] = -(-good[t // own_tiles] // BLOCK)
    seen, slots = {}, {}
    for run, is_own, tile, b0, nb, slot, row0, seq, tokens in segs[:n].tolist():
        assert nb >= 1 and b0 >= 0 and b0 + nb <= want[is_own, tile]
        for k in range(b0, b0 + nb):
            assert seen.setdefault((is_own, tile, k), run) == run
        assert (is_own, slot) not in slots, "a slot with two segments"
        slots[is_own, slot] = (tile, nb)
        # the slots the workspace has room for
        assert 0 <= slot < (batch * own_tiles if is_own else tiles) + pairs - 1
        if is_own:
            assert seq == tile // own_tiles and tokens == good[seq]
            assert row0 == (seq * q_len + tile % own_tiles * OWN_Q) * HEADS
        else:
            assert row0 == tile * ROWS
    assert len(seen) == sum(want.values()), "a block in no segment"
    for (is_own, tile), nb in want.items():
        first, count = tab[tile + (tiles if is_own else 0)].tolist()
        mine = sorted(s for (o, s), (t, _) in slots.items() if o == is_own and t == tile)
        assert mine == (list(range(first, first + count)) if nb else [])
        assert (count == 0) == (nb == 0)


@pytest.mark.parametrize("batch,q_len,pages,own,room,copied", [
    (5, 1, 1, [1, 1, 1, 1, 1], 1, True), (6, 1, 640, [3, 1200, 64, 700, 1, 1279], 1280, True),
    (1, 8, 1, [8], 8, True), (128, 1, 257, [1 + 2 * b for b in range(128)], 256, True),
    (40, 4, 37, [4 + b for b in range(40)], 64, True), (5, 1, 3, [0, 300, -5, 9999, 256], 300, True),
    (7, 1, 2, [0] * 7, 512, True), (6, 2, 4, [0, 0, 0, 0, 0, 700], 768, True),
    (6, 2, 4, [700, 0, 0, 0, 0, 0], 768, True), (32, 1, 512, [2048] * 32, 2048, False),
    (1000, 8, 3, [8] * 1000, 8, False), (16, 5, 4096, [5] * 16, 1000, True)])
@pytest.mark.parametrize("sms", [2, 3, 148, 600])
def test_plan(walk, batch, q_len, pages, own, room, copied, sms):
    check(walk, batch, q_len, pages, own, room, copied, sms)


def test_drawn_plans(walk):
    rng = random.Random(7)
    for _ in range(300):
        batch, q_len = rng.choice([1, 2, 5, 9, 30, 64, 128]), rng.randint(1, 8)
        pages, room = int(2 ** rng.uniform(0, 12)), q_len + int(2 ** rng.uniform(0, 11))
        copied = batch * -(-room // BLOCK) * BLOCK <= 1 << 15
        own = [rng.choice([rng.randint(q_len, room), q_len, room, room + 1, q_len - 1, -3]) for _ in range(batch)]
        check(walk, batch, q_len, pages, own, room, copied, rng.choice([2, 17, 148, 148, 256]))
