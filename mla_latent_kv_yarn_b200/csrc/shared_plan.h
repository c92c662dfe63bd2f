// The shared-prefix decode's plan: how its work (SharedWork) is cut into runs, which
// segments a run has, and where a tile's partial results lie.  Arithmetic alone, so
// that host code (its tests) runs the same functions as the kernels.
#pragma once

#include <cstdint>

#include "shared_prefix.h"
#include "xmla_device.cuh"

namespace xmla {

#define XMLA_PLAN_FN __host__ __device__ __forceinline__

// Own tokens of sequence b: 0 where its length leaves its new tokens outside
// its own pages (the merge reports it and zeroes its rows).
XMLA_PLAN_FN int own_tokens(const SharedParams& p, int b) {
  const int64_t len = p.seqlens[b], first = (int64_t)p.prefix_pages * kPage;
  return len >= first + p.q_len && len <= p.max_seqlen ? (int)(len - first) : 0;
}
XMLA_PLAN_FN int own_blocks(int tokens) { return (tokens + kSharedBlock - 1) / kSharedBlock; }
// Places of sequence b's own tiles.
XMLA_PLAN_FN int own_places(const SharedParams& p, int b) {
  const int nb = own_blocks(own_tokens(p, b));
  return nb > 0 ? (nb + 1) * p.own_tiles : 0;
}

// All places and runs; the own parts' share is known on the device only.
XMLA_PLAN_FN SharedWork shared_work(const SharedParams& p, int own_places) {
  SharedWork w;
  w.places = (int64_t)p.tiles * (p.blocks + 1) + own_places;
  w.runs = (int32_t)(p.pairs < w.places ? p.pairs : w.places);
  return w;
}

// Where run `run` begins.  cum: own places before each sequence, and all of them
// (batch + 1 sums; not read where the prefix has all places).
XMLA_PLAN_FN SharedRun shared_run(const SharedParams& p, const SharedWork& w, int run,
                                  const int* cum) {
  SharedRun r{0, 0, 0};
  if (run >= w.runs) return r;
  const int64_t x = w.begin(run), x_own = x - (int64_t)p.tiles * (p.blocks + 1);
  r.places = w.begin(run + 1) - x;
  if (x_own < 0) {
    r.tile = (int)(x / (p.blocks + 1));
    r.place = (int)(x % (p.blocks + 1));
  } else {  // the last sequence with cum <= x_own has that place
    int lo = 0, hi = p.batch - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (cum[mid] <= x_own) lo = mid;
      else hi = mid - 1;
    }
    const int each = (cum[lo + 1] - cum[lo]) / p.own_tiles, k = (int)x_own - cum[lo];
    r.tile = p.tiles + lo * p.own_tiles + k / each;
    r.place = k % each;
  }
  return r;
}

// Slot of the first partial of tile `tile` (the prefix's, then the own ones), and how
// many it has: one for each run from that of its first block to that of its last.
XMLA_PLAN_FN int2 shared_tile_partials(const SharedParams& p, const SharedWork& w, int tile,
                                       const int* cum) {
  int64_t first = (int64_t)tile * (p.blocks + 1);
  int nb = p.blocks, local = tile;
  if (tile >= p.tiles) {
    local = tile - p.tiles;
    const int b = local / p.own_tiles, each = (cum[b + 1] - cum[b]) / p.own_tiles;
    if (each == 0) return int2{0, 0};
    first = (int64_t)p.tiles * (p.blocks + 1) + cum[b] + (int64_t)(local - b * p.own_tiles) * each;
    nb = each - 1;
  }
  const int run0 = w.run_of(first + 1);
  return int2{run0 + local, w.run_of(first + nb) - run0 + 1};
}

// The segments of a run in order.
struct Segments {
  SharedRun at;
  // the segment
  bool is_own;
  int tile;  // of the prefix or of the own parts
  int b0;    // first block
  int n;     // blocks
  int seq, tokens;  // an own tile's sequence and its own tokens

  XMLA_PLAN_FN bool next(const SharedParams& p) {
    for (; at.places > 0; ++at.tile, at.place = 0) {
      is_own = at.tile >= p.tiles;
      tile = is_own ? at.tile - p.tiles : at.tile;
      int nb = p.blocks;
      if (is_own) {
        if (tile >= p.batch * p.own_tiles) return false;
        seq = p.own_tiles == 1 ? tile : tile >> 1;
        tokens = own_tokens(p, seq);
        nb = own_blocks(tokens);
        if (nb == 0) continue;  // a sequence of bad length has no places
      }
      if (at.place == 0) {
        at.place = 1;
        if (--at.places == 0) return false;
      }
      if (at.place > nb) continue;
      b0 = at.place - 1;
      n = nb - b0 < at.places ? nb - b0 : (int)at.places;
      at.place += n;
      at.places -= n;
      return true;
    }
    return false;
  }
  // first query row (of all rows) of the tile
  XMLA_PLAN_FN int64_t row0(const SharedParams& p) const {
    if (!is_own) return (int64_t)tile * kSharedRows;
    return ((int64_t)seq * p.q_len + (tile - seq * p.own_tiles) * kSharedOwnQ) * kHeads;
  }
  // slot of the segment's partial in run `run`
  XMLA_PLAN_FN int64_t slot(int run) const { return (int64_t)run + tile; }
};
static_assert(kSharedMaxQLen <= 2 * kSharedOwnQ, "one or two tiles per sequence");

#undef XMLA_PLAN_FN

}  // namespace xmla
