// Host-side interface of the shared-prefix kernels (shared_prefix.cu): decode
// attention of a batch whose sequences all begin with the same cache pages.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "yarn.cuh"

namespace xmla {

constexpr int kSharedMaxQLen = 8;      // new tokens per sequence and call
constexpr int kSharedRows = 128;       // query rows of a tile (64 per CTA of the pair)
constexpr int kSharedBlock = 256;      // prefix tokens of one step of a pair
constexpr int kSharedMaxPairs = 128;   // CTA pairs of the grid at most

constexpr int kSharedOwnQ = 4;         // queries of a sequence in one tile of its own part
// Own parts with room for at most this many tokens (batch * longest, rounded up to
// blocks) are copied and attended with the prefix; larger ones go through the
// split-K kernel, which reads them once.  The rule goes by room, which the host
// knows; the lengths are on the device.  Measured in us per call (replayed graph,
// every own part as long as its room), together and apart:
//   over 192 shared tokens     8 sequences x 1,536  26 / 36    24 x 1,536  44 / 41
//   over 4,096                16 x 2,048  42 / 46 (the border)
//   over 8,192                64 x 512    74 / 73 (the border)  64 x 1,024  98 / 79
//   over 16,448              128 x 333   168 / 147
//   over 32,768               32 x 512    90 / 92  x 1,024  101 / 96  x 2,048  123 / 103
constexpr int64_t kSharedOwnTokens = 1 << 15;

// Up to so many queries in all, sharing does not pay for the copy: the call runs the
// split-K kernel over each sequence's whole length, with the query as hi and lo
// parts.  It takes as long for several queries of one sequence as for as many
// sequences.  Measured in us per call (replayed graph, 300 own tokens), this way / by
// sharing, over so many shared tokens:
//   queries       64      1,024      4,096     32,768    131,072
//      1       17 / 21    19 / 21    19 / 24    23 / 46    42 / 114
//      2       18 / 22    20 / 22    20 / 24    28 / 47    60 / 114
//      4       19 / 22    21 / 22    23 / 24    39 / 46   102 / 116
//      6       21 / 23    23 / 23    26 / 26    53 / 50   149 / 139
//      8       22 / 23    24 / 23    26 / 27    64 / 50   192 / 134
constexpr int kSharedFewUnits = 4;

// Work of the attention kernel: tiles of query rows by blocks of 256 tokens.
// First the prefix's, tiles of 128 rows of the whole batch; then, sequence by
// sequence, the own parts', tiles of up to four queries of one sequence.  Laid end
// to end, a tile of nb blocks takes 1 + nb places: one for what a tile costs by
// itself (its query rows in, its sums out: about a block's time), then its blocks.
// The places are cut into runs of equal length, one per CTA pair; the blocks of a
// run that belong to one tile are a segment, with a partial result of its own at
// slot run + tile.
struct SharedWork {
  int64_t places;
  int32_t runs;  // <= places
  __host__ __device__ int64_t begin(int64_t run) const { return run * places / runs; }
  // the run that holds place f: the last one with begin(run) <= f
  __host__ __device__ int32_t run_of(int64_t f) const { return (int32_t)(((f + 1) * runs - 1) / places); }
};

// Where a run begins: tile (the prefix's, then the own ones), place within it,
// and how many places it has.
struct __align__(16) SharedRun {
  int32_t tile, place;
  int64_t places;
};

struct SharedParams {
  const __nv_bfloat16* q;        // [batch * q_len, 32, 192]
  const uint16_t* pool;          // [num_blocks, 64, 576] bf16 bits
  const int32_t* prefix_table;   // [prefix_pages]
  const int32_t* block_table;    // [batch, max_blocks]
  const int32_t* seqlens;
  __half* q16;                   // [9, rows, 64] absorbed queries, by groups of 64 columns
  __half* kv16;                  // [9, prefix tokens, 64] the prefix rows
  __half* own16;                 // [9, batch * own_pad, 64] the own rows (NULL: split-K kernel)
  float* part_o;                 // [slots, 128, 128, 4] unnormalised O of each prefix segment, by
                                 // groups of four latent columns: [column / 4][row][column % 4]
  float* part_ml;                // [slots, 128, 2] reference maximum (log2 units) and sum
  float* own_o;                  // the own parts': [slots, 128, own_rows, 4] and [slots, own_rows,
  float* own_ml;                 // 2], or, from the split-K kernel, [work items, 32, 512]
  SharedRun* run_tab;            // [pairs]
  int2* tile_tab;                // [tiles + own tiles] {slot of a tile's first partial, partials}
  __nv_bfloat16* q_ext;          // split-K kernel only: hi and lo query rows (split layout),
  int4* work_tab;                // its plan (DecodeParams::work_tab; NULL: one item per unit)
  int2* unit_tab;                // and {first work item, count} of each unit
  __nv_bfloat16* o_hi;           // [rows, 512] merged latent output, hi and lo parts
  __nv_bfloat16* o_lo;
  int32_t* status;
  uint64_t wait_limit_ns;
  int64_t num_blocks;
  int64_t max_seqlen;
  int64_t rows;                  // batch * q_len * 32
  int32_t tiles, blocks;         // of the prefix
  float qscale;                  // softmax scale * log2 e
  int32_t pairs;                 // CTA pairs of the grid
  int32_t own_pad;               // own tokens of a sequence at most, rounded up to 256
  int32_t own_tiles;             // tiles of a sequence's own part
  int32_t own_rows;              // rows of such a tile at most: 32 * min(q_len, 4)
  int32_t prefix_pages;
  int32_t max_blocks;
  int32_t batch;
  int32_t q_len;
  int32_t units;                 // batch * q_len
  int32_t items;                 // work items of the split-K kernel
};

// A table of whole sequences ([batch, cols], the prefix's blocks before the own
// ones) and the lengths, 0 where one leaves its new tokens outside its own pages.
cudaError_t launch_shared_table(const SharedParams& p, int32_t* table, int32_t cols, int32_t* lens,
                                cudaStream_t st);
// Absorbed queries (and their hi/lo rows) and the plan of the own part.  q_map:
// the query [units, 32, 192] as a 3-D map, box 64 x 1 x 128; wuk_map: W_UK as
// [4096, 512], box 64 x 128 (bf16, 128-byte swizzle).
cudaError_t launch_shared_absorb(const CUtensorMap& q_map, const CUtensorMap& wuk_map,
                                 const SharedParams& p, const RopeTable& tab, cudaStream_t st);
// The fp16 copies of the prefix rows and of the own rows.
cudaError_t launch_shared_copy(const SharedParams& p, cudaStream_t st);
// The attention of every query row over the prefix and its own tokens, as
// segments.  q_map: q16, box 64 x 64 x 9; k_map: kv16, box 64 x 128 x 1; v_map:
// kv16, box 64 x 64 x 2; ko_map, vo_map: the same of own16 (columns x rows x
// groups, 128-byte swizzle).
cudaError_t launch_shared_attn(const CUtensorMap& q_map, const CUtensorMap& k_map,
                               const CUtensorMap& v_map, const CUtensorMap& ko_map,
                               const CUtensorMap& vo_map, const SharedParams& p, cudaStream_t st);
// The latent output of every row from its segments (and its work items).
cudaError_t launch_shared_merge(const SharedParams& p, cudaStream_t st);

// The W_UV product of the latent output, to out [units, 32, 128].  hi_map, lo_map:
// o_hi and o_lo as [units, 32, 512] 3-D maps, box 64 x 1 x box_rows (the units,
// at most 128, rounded up to 8); wuv_map: W_UV as [16384, 128], box 64 x 128.
cudaError_t launch_shared_out(const CUtensorMap& hi_map, const CUtensorMap& lo_map,
                              const CUtensorMap& wuv_map, const SharedParams& p, uint32_t box_rows,
                              __nv_bfloat16* out, cudaStream_t st);

}  // namespace xmla
